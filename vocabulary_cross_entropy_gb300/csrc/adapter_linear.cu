// Low-rank adapters of many requests at once, beside a projection that they share:
//     out_n = y_n + s_i B_i (A_i x_n),   i = index[n],   A_i [r, H], B_i [V, r].
//
// Three kernels.  One sorts the tokens by their adapters, in tiles of at most 64 of one
// adapter.  The second computes t_n = A_i x_n, a tile shared by a cluster of blocks that
// divide the hidden dimension.  The third adds s_i B_i t_n to y: it reads each adapter's B
// once per tile and y once.
//
// The last one carries the work, and its bytes bound it: a token's 2 r operations per
// logit are few beside the logit's read and write (r = 64: 32 per byte, where the memory takes
// as long as 290).  So the products go through the warp-level tensor instruction with operands
// straight from global memory to registers: B is used by the warp that loads it alone, and
// staging it for the block-level instruction would cost a pass through shared memory and
// tensor memory for each logit.
//
// Precision.  t is FP32 and is multiplied as a sum of BF16 terms, three (all 24 bits) for FP32
// logits, two (16 bits: 2^-17 of the adapter's part) for BF16 logits, whose own rounding is
// 2^-9.  FP32 hidden states enter as three terms too.

#include "head_internal.cuh"
#include "sm100_ptx.cuh"

#include <algorithm>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kTile = 64;             // tokens of a tile
constexpr int kMTiles = kTile / 16;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlices = 8;            // blocks of a cluster that divide the hidden dimension
constexpr int kRankBlock = 32;        // ranks per block of the second kernel
constexpr int kVWarp = 32;            // logits per warp and step of the third
constexpr int kVBlock = kWarps * kVWarp;
constexpr int kPlanThreads = 1024;
constexpr int kMaxAdapters = VCE_MAX_ADAPTERS;

struct Tile {
    int adapter, start, count;  // adapter -1: tokens without one
};

struct Plan {
    int n_work, n_all;  // tiles with an adapter, and all
};

// ---------------------------------------------------------------------------
// the order of the tokens
// ---------------------------------------------------------------------------

struct PlanArgs {
    const int* index;
    int n, adapters, copy;  // copy: tokens without an adapter get tiles too
    Plan* plan;
    Tile* tiles;
    int* perm;
    int* dev_status;
};

__device__ __forceinline__ int2 scan(int2 v, int2* warp_sum) {  // sums of the threads up to this one
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) v.x += x, v.y += y;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int2 b = lane < warp ? warp_sum[lane] : make_int2(0, 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        b.x += __shfl_xor_sync(0xffffffffu, b.x, o);
        b.y += __shfl_xor_sync(0xffffffffu, b.y, o);
    }
    return make_int2(v.x + b.x, v.y + b.y);
}

// One block.  The order within an adapter is any: no token's result depends on its neighbours.
__global__ void __launch_bounds__(kPlanThreads) adapter_plan(const PlanArgs a) {
    __shared__ int count[kMaxAdapters + 1];  // the last: no adapter; then the places of the next tokens
    __shared__ int2 warp_sum[kPlanThreads / 32];
    const int tid = threadIdx.x;
    constexpr int kPer = kMaxAdapters / kPlanThreads;
    for (int i = tid; i <= a.adapters; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    for (int n = tid; n < a.n; n += kPlanThreads) {
        const int i = a.index[n];
        const bool has = i >= 0 && i < a.adapters;
        if (!has && i != -1) report(a.dev_status, VCE_DEVSTATUS_BAD_INDEX);
        atomicAdd(&count[has ? i : a.adapters], 1);
    }
    __syncthreads();
    int2 mine = make_int2(0, 0);  // tokens and tiles of this thread's adapters
    int c[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        c[k] = i < a.adapters ? count[i] : 0;
        mine.x += c[k], mine.y += (c[k] + kTile - 1) / kTile;
    }
    const int2 upto = scan(mine, warp_sum);
    int at = upto.x - mine.x, tile = upto.y - mine.y;
    const int none = count[a.adapters];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = tid * kPer + k;
        if (i >= a.adapters) break;
        for (int j = 0; j < c[k]; j += kTile) a.tiles[tile++] = {i, at + j, min(kTile, c[k] - j)};
        count[i] = at;
        at += c[k];
    }
    if (tid == kPlanThreads - 1) {  // the sums of all
        *a.plan = {upto.y, upto.y + (a.copy ? (none + kTile - 1) / kTile : 0)};
        if (a.copy)
            for (int j = 0; j < none; j += kTile) a.tiles[upto.y + j / kTile] = {-1, upto.x + j, min(kTile, none - j)};
        count[a.adapters] = upto.x;
    }
    __syncthreads();
    for (int n = tid; n < a.n; n += kPlanThreads) {
        const int i = a.index[n];
        const int p = atomicAdd(&count[i >= 0 && i < a.adapters ? i : a.adapters], 1);
        if (VCE_BOUNDS(p >= 0 && p < a.n, a.dev_status)) a.perm[p] = n;
    }
}

// ---------------------------------------------------------------------------
// products of 16 x 16 by 16 x 8 BF16 values
// ---------------------------------------------------------------------------

// Lane (g, q) = (lane / 4, lane % 4) holds of A rows g and g + 8, of B column g, and of C rows
// g and g + 8, columns 2 q and 2 q + 1.  The four values of k that it holds of A and of B need
// only be the same ones: four that are neighbours in memory, so that a lane loads vectors.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as a sum of BF16 terms, exactly where there are three: each term takes the leading bits of
// what is left (cut off, not rounded: rounding up could overflow); the last of two is rounded.
template <int TERMS>
__device__ __forceinline__ void split(float x, uint32_t (&t)[TERMS]) {  // BF16 bits
    float rest = x;
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        const bool last = i + 1 == TERMS;
        const uint32_t bits = __float_as_uint(rest);
        t[i] = last ? uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(rest))) : bits >> 16;
        const float d = rest - __uint_as_float(bits & 0xffff0000u);
        rest = fabsf(rest) <= 3.402823466e38f ? d : 0.f;  // (an infinity or a NaN is the first term)
    }
}

template <int TERMS>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[TERMS]) {  // pairs
    uint32_t u[TERMS], v[TERMS];
    split<TERMS>(x, u);
    split<TERMS>(y, v);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) t[i] = u[i] | v[i] << 16;
}

// ---------------------------------------------------------------------------
// t = A x
// ---------------------------------------------------------------------------

struct ShrinkArgs {
    const void* x;
    int64_t x_stride;
    const __nv_bfloat16* a;  // [adapters, rank, hidden]
    int hidden, rank, n;
    const Plan* plan;
    const Tile* tiles;
    const int* perm;
    float* t;  // [n, rank], in the order of perm
    int* dev_status;
};

// A warp takes every 64th run of 32 hidden values: sums of at most hidden / 64 products stay in
// the instruction's accumulator, what is left is added up in FP32, in a fixed order.
template <typename X>
__global__ void __launch_bounds__(kThreads) adapter_shrink(const ShrinkArgs a) {
    constexpr int TERMS = sizeof(X) == 2 ? 1 : 3;
    extern __shared__ __align__(16) float red[];  // [warps][tile][kRankBlock]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int slice = int(cluster_ctarank());
    cudaGridDependencySynchronize();
    const int id = int(blockIdx.x) / kSlices;
    if (id >= a.plan->n_work) return;  // the whole cluster
    const Tile tile = a.tiles[id];
    const int r0 = int(blockIdx.y) * kRankBlock, mtiles = (tile.count + 15) / 16;

    const X* row[kMTiles][2];
#pragma unroll
    for (int m = 0; m < kMTiles; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = m * 16 + h * 8 + g;
            row[m][h] = p < tile.count ? static_cast<const X*>(a.x) + a.perm[tile.start + p] * a.x_stride : nullptr;
        }
    float c[kMTiles][kRankBlock / 8][4] = {};
    const __nv_bfloat16* const base = a.a + (int64_t(tile.adapter) * a.rank + r0) * a.hidden;
    for (int k = (slice * kWarps + warp) * 32 + q * 8; k - q * 8 < a.hidden; k += kSlices * kWarps * 32) {
        uint4 b[kRankBlock / 8];
#pragma unroll
        for (int j = 0; j < kRankBlock / 8; ++j) {
            b[j] = make_uint4(0, 0, 0, 0);
            if (k < a.hidden && r0 + j * 8 + g < a.rank &&
                VCE_BOUNDS(aligned16(base + k) && k + 8 <= a.hidden, a.dev_status))
                b[j] = __ldg(reinterpret_cast<const uint4*>(base + int64_t(j * 8 + g) * a.hidden + k));
        }
#pragma unroll
        for (int m = 0; m < kMTiles; ++m) {
            if (m >= mtiles) break;
            uint32_t x[TERMS][2][4];  // term, half of the run, operand words
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (TERMS == 1) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (k < a.hidden && row[m][h] && VCE_BOUNDS(aligned16(row[m][h] + k), a.dev_status))
                        v = __ldg(reinterpret_cast<const uint4*>(row[m][h] + k));
                    x[0][0][h] = v.x, x[0][0][2 + h] = v.y, x[0][1][h] = v.z, x[0][1][2 + h] = v.w;
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (k < a.hidden && row[m][h] && VCE_BOUNDS(aligned16(row[m][h] + k), a.dev_status))
                            v = __ldg(reinterpret_cast<const float4*>(row[m][h] + k) + s);
                        uint32_t lo[TERMS], hi[TERMS];
                        split2<TERMS>(v.x, v.y, lo);
                        split2<TERMS>(v.z, v.w, hi);
#pragma unroll
                        for (int i = 0; i < TERMS; ++i) x[i][s][h] = lo[i], x[i][s][2 + h] = hi[i];
                    }
                }
            }
#pragma unroll
            for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
                for (int j = 0; j < kRankBlock / 8; ++j) {
                    mma(c[m][j], x[i][0], b[j].x, b[j].y);
                    mma(c[m][j], x[i][1], b[j].z, b[j].w);
                }
        }
    }
    const int entries = mtiles * 16 * kRankBlock;
#pragma unroll
    for (int m = 0; m < kMTiles; ++m) {
        if (m >= mtiles) break;
#pragma unroll
        for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(&red[warp * (kTile * kRankBlock) + (m * 16 + h * 8 + g) * kRankBlock + j * 8 + 2 * q]) =
                    make_float2(c[m][j][2 * h], c[m][j][2 * h + 1]);
    }
    __syncthreads();
    for (int e = tid; e < entries; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w * (kTile * kRankBlock) + e];
        red[e] = s;
    }
    cluster_sync();
    const int share = entries / kSlices;  // entries are a multiple of 512
    for (int e = slice * share + tid; e < (slice + 1) * share; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&red[e]), k)) : "memory");
            s += v;
        }
        const int p = e / kRankBlock, r = r0 + e % kRankBlock;
        if (p < tile.count && r < a.rank) a.t[int64_t(tile.start + p) * a.rank + r] = s;
    }
    cluster_sync();  // nobody leaves while its shared memory is read
}

// ---------------------------------------------------------------------------
// out = y + s B t
// ---------------------------------------------------------------------------

struct ExpandArgs {
    const __nv_bfloat16* b;  // [adapters, vocab, rank]
    const float* scale;
    const float* t;
    const void* y;
    void* out;
    int64_t y_stride, out_stride;
    int vocab, rank, n;
    int vectors;  // rows start at 16-byte boundaries
    const Plan* plan;
    const Tile* tiles;
    const int* perm;
    int* dev_status;
};

template <typename Y>
struct Eight;  // eight neighbouring logits of a row
template <>
struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
    __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ static uint32_t sum(uint32_t a, float x, float y) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(a << 16) + x, __uint_as_float(a & 0xffff0000u) + y);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    __device__ __forceinline__ void add(int i, float x, float y) {  // to the pair 2 i, 2 i + 1
        uint32_t& a = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
        a = sum(a, x, y);
    }
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
        uint32_t u[4] = {};
        const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) u[i / 2] |= uint32_t(s[i]) << (i % 2 * 16);
        w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void store_some(__nv_bfloat16* p, int n) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        unsigned short* s = reinterpret_cast<unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) s[i] = static_cast<unsigned short>(u[i / 2] >> (i % 2 * 16));
    }
};
template <>
struct Eight<float> {
    float v[8];
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ __forceinline__ void add(int i, float x, float y) { v[2 * i] += x, v[2 * i + 1] += y; }
    __device__ __forceinline__ void load_some(const float* p, int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    }
    __device__ __forceinline__ void store_some(float* p, int n) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
};

// The first of the four neighbouring ranks that lane q holds in step s of KS.
template <int KS>
__device__ __forceinline__ int rank_of(int s, int q) { return KS == 1 ? 4 * q : 32 * (s / 2) + 8 * q + 4 * (s & 1); }

// Tokens are the rows of the products and logits the columns: column 2 q + e of tile j is logit
// 8 q + 2 j + e of the warp's 32, so that a lane ends up with eight neighbours of a row.
template <typename Y, int KS>
__global__ void __launch_bounds__(kThreads) adapter_expand(const ExpandArgs a) {
    constexpr int TERMS = sizeof(Y) == 2 ? 2 : 3;
    extern __shared__ __align__(16) uint4 frag[];  // [TERMS][kMTiles][KS][32]: operands of t
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    cudaGridDependencySynchronize();
    const int vblocks = (a.vocab + kVBlock - 1) / kVBlock;
    const int64_t units = int64_t(a.plan->n_all) * vblocks;
    const int64_t first = units * blockIdx.x / gridDim.x, last = units * (blockIdx.x + 1) / gridDim.x;
    int id = -1;
    Tile tile{};
    int64_t token[kMTiles][2];
    for (int64_t unit = first; unit < last; ++unit) {
        const int now = int(unit / vblocks);
        if (now != id) {
            id = now;
            tile = a.tiles[id];
            const float scale = tile.adapter >= 0 && a.scale ? a.scale[tile.adapter] : 1.f;
            __syncthreads();
            if (tile.adapter >= 0)
                for (int i = tid; i < kMTiles * KS * 32; i += kThreads) {
                    const int l = i & 31, s = i / 32 % KS, m = i / (32 * KS), r = rank_of<KS>(s, l & 3);
                    float4 v[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int p = m * 16 + h * 8 + (l >> 2);
                        v[h] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (p < tile.count && r < a.rank)
                            v[h] = *reinterpret_cast<const float4*>(a.t + int64_t(tile.start + p) * a.rank + r);
                    }
                    uint32_t w[4][TERMS];
                    split2<TERMS>(v[0].x * scale, v[0].y * scale, w[0]);
                    split2<TERMS>(v[1].x * scale, v[1].y * scale, w[1]);
                    split2<TERMS>(v[0].z * scale, v[0].w * scale, w[2]);
                    split2<TERMS>(v[1].z * scale, v[1].w * scale, w[3]);
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) frag[k * (kMTiles * KS * 32) + i] = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
                }
#pragma unroll
            for (int m = 0; m < kMTiles; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = m * 16 + h * 8 + g;
                    token[m][h] = p < tile.count ? a.perm[tile.start + p] : -1;
                }
            __syncthreads();
        }
        const int v0 = int(unit - int64_t(id) * vblocks) * kVBlock + warp * kVWarp;
        if (v0 >= a.vocab) continue;
        uint32_t b[4][KS][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int v = v0 + 8 * (g >> 1) + 2 * j + (g & 1);
            const __nv_bfloat16* const at = a.b + (int64_t(tile.adapter) * a.vocab + v) * a.rank;
            const bool ok = tile.adapter >= 0 && v < a.vocab;
            if constexpr (KS == 1) {
                uint2 w = make_uint2(0, 0);
                if (ok && 4 * q < a.rank && VCE_BOUNDS((reinterpret_cast<uintptr_t>(at) & 7) == 0, a.dev_status))
                    w = __ldg(reinterpret_cast<const uint2*>(at + 4 * q));
                b[j][0][0] = w.x, b[j][0][1] = w.y;
            } else {
#pragma unroll
                for (int s = 0; s < KS; s += 2) {
                    const int r = rank_of<KS>(s, q);
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (ok && r < a.rank && VCE_BOUNDS(aligned16(at + r), a.dev_status))
                        w = __ldg(reinterpret_cast<const uint4*>(at + r));
                    b[j][s][0] = w.x, b[j][s][1] = w.y, b[j][s + 1][0] = w.z, b[j][s + 1][1] = w.w;
                }
            }
        }
        const int v = v0 + 8 * q, left = a.vocab - v;  // this lane's eight logits
        const bool whole = a.vectors && left >= 8;
        auto fetch = [&](Eight<Y>& e, int64_t n) {
            e.clear();
            if (n < 0 || left <= 0) return;
            const Y* const p = static_cast<const Y*>(a.y) + n * a.y_stride + v;
            if (whole) e.load(p);
            else e.load_some(p, left);
        };
        Eight<Y> e[2];
        fetch(e[0], token[0][0]);
        fetch(e[1], token[0][1]);
#pragma unroll
        for (int m = 0; m < kMTiles; ++m) {
            if (m * 16 >= tile.count) break;
            Eight<Y> next[2];
            if (m + 1 < kMTiles) {  // on their way while this tile is multiplied
                fetch(next[0], token[m + 1 < kMTiles ? m + 1 : m][0]);
                fetch(next[1], token[m + 1 < kMTiles ? m + 1 : m][1]);
            }
            float c[4][4] = {};
            if (tile.adapter >= 0) {
#pragma unroll
                for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        const uint4 f = frag[((k * kMTiles + m) * KS + s) * 32 + lane];
                        const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma(c[j], w, b[j][s][0], b[j][s][1]);
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = token[m][h];
                if (n >= 0 && left > 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[h].add(j, c[j][2 * h], c[j][2 * h + 1]);
                    Y* const p = static_cast<Y*>(a.out) + n * a.out_stride + v;
                    if (whole) e[h].store(p);
                    else e[h].store_some(p, left);
                }
                e[h] = next[h];
            }
        }
    }
}

template <typename Y>
auto expand_kernel(int ks) {
    return ks == 1 ? adapter_expand<Y, 1> : ks == 2 ? adapter_expand<Y, 2> : ks == 4 ? adapter_expand<Y, 4> : adapter_expand<Y, 8>;
}

struct Carved {
    Plan* plan;
    Tile* tiles;
    int* perm;
    float* t;
    size_t bytes;
};

int64_t most_tiles(int64_t n, int64_t adapters) { return std::min(n, adapters + 1) + n / kTile; }

Carved carve(void* ws, int64_t n, int64_t adapters, int rank) {
    char* p = static_cast<char*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* r = p + at;
        at += align256(bytes);
        return r;
    };
    Carved c{};
    c.plan = reinterpret_cast<Plan*>(take(sizeof(Plan)));
    c.tiles = reinterpret_cast<Tile*>(take(size_t(most_tiles(n, adapters)) * sizeof(Tile)));
    c.perm = reinterpret_cast<int*>(take(size_t(n) * 4));
    c.t = reinterpret_cast<float*>(take(size_t(n) * rank * 4));
    c.bytes = at;
    return c;
}

}  // namespace

size_t adapter_ws_bytes(int64_t n, int64_t adapters, int rank) {
    static char none;
    return carve(&none, n, adapters, rank).bytes;
}

vce_status launch_adapter_linear(const void* y, int y_dtype, int64_t n, int64_t vocab, int64_t y_stride, const void* x,
                                 int x_dtype, int64_t hidden, int64_t x_stride, const void* a, const void* b,
                                 int64_t adapters, int rank, const int* index, const float* scale, void* out,
                                 int64_t out_stride, void* ws, int* dev_status, cudaStream_t s, const DeviceInfo& dev) {
    if (n == 0) return VCE_OK;
    const Carved w = carve(ws, n, adapters, rank);
    const bool in_place = out == y;
    const PlanArgs pa{index, int(n), int(adapters), !in_place, w.plan, w.tiles, w.perm, dev_status};
    count_launch();
    adapter_plan<<<1, kPlanThreads, 0, s>>>(pa);
    if (cudaGetLastError() != cudaSuccess) return VCE_ERR_CUDA;

    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSlices;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;

    const ShrinkArgs sa{x, x_stride, static_cast<const __nv_bfloat16*>(a), int(hidden), rank, int(n), w.plan, w.tiles,
                        w.perm, w.t, dev_status};
    auto shrink = x_dtype == VCE_BF16 ? adapter_shrink<__nv_bfloat16> : adapter_shrink<float>;
    const size_t shrink_smem = size_t(kWarps) * kTile * kRankBlock * 4;
    const int ks = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
    auto expand = y_dtype == VCE_BF16 ? expand_kernel<__nv_bfloat16>(ks) : expand_kernel<float>(ks);
    const size_t expand_smem = size_t(y_dtype == VCE_BF16 ? 2 : 3) * kMTiles * ks * 32 * sizeof(uint4);
    static std::mutex mu;
    static bool ready[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev.ordinal]) {
            for (auto k : {adapter_shrink<__nv_bfloat16>, adapter_shrink<float>})
                if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shrink_smem)) != cudaSuccess)
                    return VCE_ERR_CUDA;
            ready[dev.ordinal] = true;
        }
    }
    cfg.gridDim = dim3(unsigned(std::min(n, adapters) + n / kTile) * kSlices, unsigned((rank + kRankBlock - 1) / kRankBlock));
    cfg.dynamicSmemBytes = shrink_smem;
    cfg.numAttrs = 2;
    count_launch();
    if (cudaLaunchKernelEx(&cfg, shrink, sa) != cudaSuccess) return VCE_ERR_CUDA;

    const int es = y_dtype == VCE_BF16 ? 2 : 4;
    const bool vectors = reinterpret_cast<uintptr_t>(y) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                         (n == 1 || (y_stride * es % 16 == 0 && out_stride * es % 16 == 0));
    const ExpandArgs ea{static_cast<const __nv_bfloat16*>(b), scale, w.t, y, out, y_stride, out_stride, int(vocab), rank,
                        int(n), vectors, w.plan, w.tiles, w.perm, dev_status};
    const int64_t vblocks = (vocab + kVBlock - 1) / kVBlock;
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(most_tiles(n, adapters) * vblocks, int64_t(dev.num_sms) * 4)));
    cfg.dynamicSmemBytes = expand_smem;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, expand, ea) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
