// Low-rank adapters of many requests at once, beside a projection that they share:
//     out_n = y_n + s_i B_i (A_i x_n),   i = index[n],   A_i [r, H], B_i [V, r].
//
// Three kernels.  One sorts the tokens by their adapters, in tiles of at most 64 of one
// adapter (few tokens are sorted by each block of the second).  The second computes t_n = A_i x_n, a
// tile shared by a cluster of blocks that divide the hidden dimension.  The third adds s_i B_i t_n to y: it reads each adapter's B
// once per tile and y once.  Each starts while the one before still runs, up to its wait for it.
//
// The last one carries the work, and its bytes are the floor: a token's 2 r operations per
// logit are few beside the logit's read and write (r = 64: 32 per byte, where the memory takes
// as long as 290).  So the products go through the warp-level tensor instruction, whose results
// lie in the registers of the lanes that hold the logits; the block-level one would take each logit
// through tensor memory as well.  There are two forms of it: adapter_expand_few for much work of few tokens
// per adapter and small ranks, adapter_expand_many for the others.  They add the same products in the same order, and
// a token's result does not depend on which one takes it.
//
// Precision.  t is FP32 and is multiplied as a sum of BF16 terms, three (all 24 bits) for FP32
// logits, two (2^-17 of the adapter's part) for BF16 logits, whose own rounding is
// 2^-8.  FP32 hidden states enter as three terms too.

#include "head_internal.cuh"
#include "sm100_ptx.cuh"

#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

namespace vce {
namespace {

using namespace sm100;

constexpr int kTile = 64;             // tokens of a tile
constexpr int kMTiles = kTile / 16;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlices = 8;            // blocks of a cluster that divide the hidden dimension, at most
constexpr int kSelf = 128;            // tokens up to which each block of the second kernel sorts them by itself: 256 with 64
                                      // adapters, 128256 logits took 96.6 us so, 92.6 by adapter_plan; with 16 adapters equal
constexpr int kRankBlock = 32;        // ranks per block of the second kernel
constexpr int kVWarp = 32;            // logits of a warp, and
constexpr int kVBlock = kWarps * kVWarp;  // of a block of adapter_expand_many
constexpr int kRun = 512;             // logits of a unit that is handed out, or a multiple
constexpr int kMaxStages = 6;         // of adapter_expand_few's ring
constexpr int kRingBytes = 216 << 10;
constexpr int64_t kMany = 24;         // tokens per adapter (of the table: the host does not know which are used) from which
                                      // adapter_expand_many takes them, and
constexpr int kShort = 13, kShortAny = 7;  // units of its work per block up to which it does (any alignment)
constexpr int kMulWarps = 16;         // warps of adapter_expand_few that multiply
constexpr int kCellPitch = 292;       // floats: a row of kVBlock products, one unused behind every eight (no bank conflicts)
constexpr int kMaxBlock = 1024;       // logits of a stage, at most
constexpr int kStageRows = 32 << 10;  // bytes of y in a stage, and
constexpr int kStageB = 32 << 10;     // of B, at most
constexpr int kPlanThreads = 1024;
constexpr int kMaxAdapters = VCE_MAX_ADAPTERS;

struct Tile {
    int adapter, start, count;  // adapter -1: tokens without one
};

struct Plan {
    int n_work, n_all;  // tiles with an adapter, and all
    int next;           // the next unit of work of the third kernel
};

// ---------------------------------------------------------------------------
// the order of the tokens
// ---------------------------------------------------------------------------

struct PlanArgs {
    const int* index;
    int n, adapters, copy;  // copy: tokens without an adapter get tiles too
    int tiles_cap;          // how many tiles there is room for
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
    cudaTriggerProgrammaticLaunchCompletion();  // the next kernel starts, up to its wait for this one
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
        for (int j = 0; j < c[k]; j += kTile, ++tile)
            if (VCE_BOUNDS(tile < a.tiles_cap, a.dev_status)) a.tiles[tile] = {i, at + j, min(kTile, c[k] - j)};
        count[i] = at;
        at += c[k];
    }
    if (tid == kPlanThreads - 1) {  // the sums of all
        *a.plan = {upto.y, upto.y + (a.copy ? (none + kTile - 1) / kTile : 0), 0};
        if (a.copy)
            for (int j = 0; j < none; j += kTile)
                if (VCE_BOUNDS(upto.y + j / kTile < a.tiles_cap, a.dev_status))
                    a.tiles[upto.y + j / kTile] = {-1, upto.x + j, min(kTile, none - j)};
        count[a.adapters] = upto.x;
    }
    __syncthreads();
    for (int n = tid; n < a.n; n += kPlanThreads) {
        const int i = a.index[n];
        const int p = atomicAdd(&count[i >= 0 && i < a.adapters ? i : a.adapters], 1);
        if (VCE_BOUNDS(p >= 0 && p < a.n, a.dev_status)) a.perm[p] = n;
    }
}

// The token at a place of the order.
__device__ __forceinline__ int token_at(const int* perm, int at, int n, int* dev_status) {
    if (!VCE_BOUNDS(at >= 0 && at < n, dev_status)) return 0;
    const int token = perm[at];
    return VCE_BOUNDS(token >= 0 && token < n, dev_status) ? token : 0;
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

__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  // c = the product
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
        rest = fabsf(rest) == INFINITY ? 0.f : d;  // (a NaN's later terms are NaN: its first one's bits may be an infinity's)
    }
}

// Pairs.  The first of two terms is rounded, too, where it cannot overflow: 2^-17 of x is left at most (2^-16 if it were
// cut off).
template <int TERMS>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[TERMS]) {
    if constexpr (TERMS == 2) {
        if (fmaxf(fabsf(x), fabsf(y)) < 0x1.ffp127f) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
            t[0] = *reinterpret_cast<const uint32_t*>(&a);
            const __nv_bfloat162 b = __floats2bfloat162_rn(x - __uint_as_float(t[0] << 16), y - __uint_as_float(t[0] & 0xffff0000u));
            t[1] = *reinterpret_cast<const uint32_t*>(&b);
            return;
        }
    }
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
    PlanArgs plan_args;
    int slices;  // blocks of a cluster
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

// The order of up to kSelf tokens, which every block finds for itself: a token's place is the number of those
// before it.  The first block leaves it to the next kernel.  Returns this block's tile (count 0: none).
struct Sorted {
    int key[kSelf], sorted[kSelf], order[kSelf];
    uint32_t starts[kSelf / 32];  // a bit for each place at which a tile starts
    int none;                     // tokens without an adapter, which come last
    Tile tile;
};

__device__ __forceinline__ Tile plan_here(const PlanArgs& a, Sorted& sh, int id, bool first) {
    const int tid = threadIdx.x;
    int adapter = 0;
    if (tid < a.n) {
        adapter = a.index[tid];
        if (adapter < 0 || adapter >= a.adapters) {
            if (adapter != -1 && first) report(a.dev_status, VCE_DEVSTATUS_BAD_INDEX);
            adapter = a.adapters;
        }
    }
    const int low = adapter * kSelf, mine = low + tid;
    if (tid < kSelf) sh.key[tid] = tid < a.n ? mine : INT_MAX;
    if (tid < kSelf / 32) sh.starts[tid] = 0;
    if (tid == 0) sh.none = 0, sh.tile.count = 0;
    __syncthreads();
    int place = 0, less = 0, same = 0;
    if (tid < a.n) {
        for (int j = 0; j < a.n; j += 4) {  // (what is behind the last token is above every key)
            const int4 k = *reinterpret_cast<const int4*>(&sh.key[j]);
            place += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
        }
        sh.sorted[place] = mine;
    }
    __syncthreads();
    if (tid < a.n) {
        auto below = [&](int key) {  // how many keys are
            int at = 0;
#pragma unroll
            for (int step = kSelf / 2; step > 0; step /= 2)
                if (at + step <= a.n && sh.sorted[at + step - 1] < key) at += step;
            return at + (at < a.n && sh.sorted[at] < key);
        };
        less = below(low), same = below(low + kSelf) - less;
        sh.order[place] = tid;
        if ((place - less) % kTile == 0) atomicOr(&sh.starts[place / 32], 1u << place % 32);
        if (adapter == a.adapters && place == less) sh.none = same;
    }
    __syncthreads();
    if (tid < a.n && (place - less) % kTile == 0) {
        int which = __popc(sh.starts[place / 32] & ((1u << place % 32) - 1));
        for (int w = 0; w < place / 32; ++w) which += __popc(sh.starts[w]);
        const bool has = adapter < a.adapters;
        const Tile tile{has ? adapter : -1, place, min(kTile, same - (place - less))};
        if (has && which == id) sh.tile = tile;
        if (first && (has || a.copy) && VCE_BOUNDS(which < a.tiles_cap, a.dev_status)) a.tiles[which] = tile;
    }
    if (first) {
        if (tid < a.n) a.perm[place] = tid;
        if (tid == 0) {
            int all = 0;
            for (uint32_t w : sh.starts) all += __popc(w);
            const int none = (sh.none + kTile - 1) / kTile;
            *a.plan = {all - none, a.copy ? all : all - none, 0};
        }
    }
    __syncthreads();
    return sh.tile;
}

// Sums of the products of every (8 slices)-th run of 32 hidden values stay in the instruction's accumulator, what is
// left is added up in FP32, in an order that the hidden dimension alone determines.
template <typename X, bool SELF>
__global__ void __launch_bounds__(kThreads, 2) adapter_shrink(const ShrinkArgs a) {
    constexpr int TERMS = sizeof(X) == 2 ? 1 : 3;
    extern __shared__ __align__(16) float red[];  // [warps][tile][kRankBlock]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int slice = int(cluster_ctarank());
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const int id = int(blockIdx.x) / a.slices;
    Tile tile;
    __shared__ __align__(16) char sorted_mem[SELF ? sizeof(Sorted) : 16];
    Sorted& sorted = *reinterpret_cast<Sorted*>(sorted_mem);
    if constexpr (SELF) {
        tile = plan_here(a.plan_args, sorted, id, blockIdx.x == 0 && blockIdx.y == 0);
        if (tile.count == 0) return;  // the whole cluster
    } else {
        if (id >= a.plan->n_work) return;
        tile = a.tiles[id];
    }
    auto token = [&](int p) { return SELF ? sorted.order[tile.start + p] : token_at(a.perm, tile.start + p, a.n, a.dev_status); };
    const int r0 = int(blockIdx.y) * kRankBlock, mtiles = (tile.count + 15) / 16;

    // The runs of 32 hidden values (slice kWarps + c), and every (slices kWarps)-th after it, are chain c of the slice,
    // one sum.  The warps divide the groups of 16 tokens and, for each, the chains.
    const int across = mtiles > 2 ? 4 : mtiles;  // warps across the tokens
    const int m = warp % across, kw = warp / across, per = kWarps / across;
    const int stride = a.slices * kWarps * 32, runs = (a.hidden + stride - 1) / stride;  // of a chain
    const int items = m < mtiles ? kWarps / per * runs : 0;
    const X* row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int p = m * 16 + h * 8 + g;
        row[h] = p < tile.count ? static_cast<const X*>(a.x) + token(p) * a.x_stride : nullptr;
    }
    const __nv_bfloat16* const base = a.a + (int64_t(tile.adapter) * a.rank + r0) * a.hidden;
    struct Item {
        uint4 b[kRankBlock / 8], x[2][sizeof(X) / 2];
    };
    constexpr int kItems = TERMS == 1 ? 3 : 2;  // on their way
    Item item[kItems];
    int chain = kw, run = 0;  // of the next item to load
    auto load = [&](Item& it) {
        const int k = (slice * kWarps + chain) * 32 + run * stride + q * 8;
        const bool in = chain < kWarps && k < a.hidden && items > 0;
#pragma unroll
        for (int j = 0; j < kRankBlock / 8; ++j) {
            it.b[j] = make_uint4(0, 0, 0, 0);
            if (in && r0 + j * 8 + g < a.rank && VCE_BOUNDS(aligned16(base + k) && k + 8 <= a.hidden, a.dev_status))
                it.b[j] = __ldg(reinterpret_cast<const uint4*>(base + int64_t(j * 8 + g) * a.hidden + k));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < int(sizeof(X)) / 2; ++i) {
                it.x[h][i] = make_uint4(0, 0, 0, 0);
                if (in && row[h] && VCE_BOUNDS(aligned16(row[h] + k), a.dev_status))
                    it.x[h][i] = __ldg(reinterpret_cast<const uint4*>(row[h] + k) + i);
            }
        if (++run == runs) run = 0, chain += per;
    };
    float c[kRankBlock / 8][4] = {};
#pragma unroll
    for (int i = 0; i < kItems; ++i) load(item[i]);
    for (int done = 0, left = runs, to = kw; done < items;) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (done >= items) break;
            Item& it = item[i];
            uint32_t x[TERMS][2][4];  // term, half of the run, operand words
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (TERMS == 1) {
                    const uint4 v = it.x[h][0];
                    x[0][0][h] = v.x, x[0][0][2 + h] = v.y, x[0][1][h] = v.z, x[0][1][2 + h] = v.w;
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint4 v = it.x[h][s];
                        uint32_t lo[TERMS], hi[TERMS];
                        split2<TERMS>(__uint_as_float(v.x), __uint_as_float(v.y), lo);
                        split2<TERMS>(__uint_as_float(v.z), __uint_as_float(v.w), hi);
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) x[t][s][h] = lo[t], x[t][s][2 + h] = hi[t];
                    }
                }
            }
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
                for (int j = 0; j < kRankBlock / 8; ++j) {
                    mma(c[j], x[t][0], it.b[j].x, it.b[j].y);
                    mma(c[j], x[t][1], it.b[j].z, it.b[j].w);
                }
            load(it);
            ++done;
            if (--left == 0) {  // the chain's sum is complete
#pragma unroll
                for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        *reinterpret_cast<float2*>(&red[to * (kTile * kRankBlock) + (m * 16 + h * 8 + g) * kRankBlock + j * 8 + 2 * q]) =
                            make_float2(c[j][2 * h], c[j][2 * h + 1]);
                        c[j][2 * h] = c[j][2 * h + 1] = 0.f;
                    }
                left = runs, to += per;
            }
        }
    }
    const int entries = mtiles * 16 * kRankBlock;
    __syncthreads();
    for (int e = tid; e < entries; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w * (kTile * kRankBlock) + e];
        red[e] = s;
    }
    cluster_sync();
    const int share = entries / a.slices;  // entries are a multiple of 512
    for (int e = slice * share + tid; e < (slice + 1) * share; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) {
            if (k >= a.slices) break;
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&red[e]), k)) : "memory");
            s += v;
        }
        const int p = e / kRankBlock, r = r0 + e % kRankBlock;
        if (p < tile.count && r < a.rank && VCE_BOUNDS(tile.start + p < a.n, a.dev_status))
            a.t[int64_t(tile.start + p) * a.rank + r] = s;
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
    int n, vocab, rank;
    int stages, stage_bytes, y_bytes, b_bytes;  // of the ring; of a stage, of its rows of y, of its part of B
    int block[4];                      // logits of a stage, by class_of a tile
    Plan* plan;
    const Tile* tiles;
    const int* perm;
    int* dev_status;
};

// The first of the four neighbouring ranks that lane q holds in step s of KS.
template <int KS>
__device__ __forceinline__ int rank_of(int s, int q) { return KS == 1 ? 4 * q : 32 * (s / 2) + 8 * q + 4 * (s & 1); }

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Four neighbouring logits at an address that is a multiple of their size.
__device__ __forceinline__ void load4(float (&x)[4], const float* p) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
}
__device__ __forceinline__ void load4(float (&x)[4], const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Tiles by how many tokens they have: up to 4, 16, 32, 64.
__host__ __device__ __forceinline__ int class_of(int count) { return count > 32 ? 3 : count > 16 ? 2 : count > 4 ? 1 : 0; }

struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int4 what[kMaxStages];  // 0 (-1: the end), first logit, number of logits, whether its tile is another one
    int abort;
};

// What the multiplying warps have to know of a tile, beside t.
template <typename Y>
struct TileInfo {
    int adapter, count;
    float scale;
    Y* out[kTile];   // the tokens' rows
    int off[kTile];  // bytes of y's rows behind a 16-byte boundary
};

// Tiles of few tokens, where there are many or many logits, and ranks up to 32.  Logits are the rows of the
// products (16) and tokens the columns (8): a tile of one token costs no more than one of eight.  A warp takes 16
// tokens and 32 logits at a time; what warps the tokens leave divide the logits.  A further warp copies y's rows and B,
// some logits at a time, through a ring in shared memory, and with a tile's first logits t and what else belongs to the
// tile.  Units of work are handed out by a counter, the larger ones first: tiles differ by a factor of 64.
//
// Rows that start off 16-byte boundaries are copied with what shares their first and last 16 bytes, except
// at a row's ends, whose odd elements are copied one by one; results go back through shared memory, so
// that a warp writes neighbours of one row.
//
// 64 tokens with 35 adapters of rank 16, 128256 FP32 logits: 47 us (4.3 TB/s), of which the copies alone take
// 40; the others are the multiplying warps' instructions, about 160 for 32 logits of a token.  256 tokens with 64
// adapters, rank 16, BF16, all three kernels, this form / the other one: 128256 logits 85 / 150 us, 128257
// (rows off 16-byte boundaries) 124 / 207.  Before the ring carried t and the tiles, each warp waited for a chain of three
// loads with each tile: 91 and 129.
//
// What bounds it for larger tiles is its copies, one for each row and stage: 66 cycles each.  Larger ranks are the other
// one's because t's operands no longer fit this one's registers (rank 64, the same: 407 / 225).
template <typename Y, int KS, bool VEC>
__global__ void __launch_bounds__(kMulWarps * 32 + 32, 1) adapter_expand_few(const __grid_constant__ ExpandArgs a) {
    constexpr int TERMS = sizeof(Y) == 2 ? 2 : 3, ES = int(sizeof(Y));
    extern __shared__ __align__(128) uint8_t smem[];  // stages: rows of y, then B, then t
    __shared__ Ring ring;
    __shared__ TileInfo<Y> infos[kMaxStages];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&ring.full[i], 32);
            mbar_init(&ring.empty[i], kMulWarps);
        }
        fence_mbar_init();
        ring.abort = 0;
    }
    __syncthreads();
    cudaGridDependencySynchronize();
    int stage = 0;
    bool ok = true;
    if (warp == kMulWarps) {
        // Unit u: a run of logits of tile tiles - 1 - u / runs (those without an adapter come first).
        const int tiles = a.plan->n_all;
        // Three to five units for each block: a unit costs a chain of loads, which few tokens' work does not cover.
        const int share = 3 + min(a.n / max(tiles, 1), 16) / 6;
        const int run = kRun * int(max(int64_t(1), min(int64_t(16), int64_t(tiles) * a.vocab / (int64_t(gridDim.x) * share * kRun))));
        const int runs = (a.vocab + run - 1) / run;
        const int64_t units = int64_t(tiles) * runs;
        int issued = 0, block = 0, pitch = 0;
        uint32_t parity = 1;  // of the ring's previous round, which the first one need not wait for
        Tile tile{};
        float scale = 1.f;
        int64_t token[2] = {-1, -1};  // this lane's
        uintptr_t row[2] = {0, 0};    // 0: none
        bool fresh = false;           // the tile's first logits are still to come
        asm volatile("fence.proxy.async.global;" ::: "memory");  // t was written by ordinary stores, and is copied from here
        auto take = [&]() { return lane == 0 ? atomicAdd(&a.plan->next, 1) : 0; };
        auto enter = [&](const Tile& t) {
            tile = t, fresh = true;
            block = a.block[class_of(tile.count)], pitch = block * ES + 32;
            scale = a.scale && tile.adapter >= 0 ? a.scale[tile.adapter] : 1.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int p = lane + 32 * h;
                token[h] = p < tile.count ? token_at(a.perm, tile.start + p, a.n, a.dev_status) : -1;
                row[h] = p < tile.count ? reinterpret_cast<uintptr_t>(static_cast<const Y*>(a.y) + token[h] * a.y_stride) : 0;
            }
        };
        // The next unit is known while one is copied, and the one after it on its way.
        int unit = __shfl_sync(0xffffffffu, take(), 0);
        int coming = take();
        if (unit < units) enter(a.tiles[tiles - 1 - unit / runs]);
        for (;;) {
            const bool end = unit >= units;
            const int next = end ? unit : __shfl_sync(0xffffffffu, coming, 0);
            if (!end) coming = take();
            const bool other = next < units && next / runs != unit / runs;
            Tile next_tile{};
            if (other) next_tile = a.tiles[tiles - 1 - next / runs];
            const int v0 = end ? 0 : unit % runs * run, v1 = end ? 1 : min(v0 + run, a.vocab);
            for (int v = v0; v < v1; v += end ? 1 : block) {
                if (issued >= a.stages) {
                    ok = mbar_wait(&ring.empty[stage], parity, &ring.abort, kPipeTimeoutNs);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                const int ve = min(v + block, v1);
                uint8_t* const to = smem + size_t(stage) * a.stage_bytes;
                uintptr_t from[2] = {0, 0};
                uint32_t bytes[2] = {0, 0}, b_bytes = 0, t_bytes = 0;
                const bool first = fresh && !end;
                if (!end) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (row[h] == 0) continue;
                        const uintptr_t s = row[h] + int64_t(v) * ES, e = row[h] + int64_t(ve) * ES, low = s & ~uintptr_t(15);
                        uintptr_t f = low, l = (e + 15) & ~uintptr_t(15);
                        if (f < row[h]) f += 16;
                        if (l > row[h] + int64_t(a.vocab) * ES) l -= 16;
                        if (f > l) f = l;
                        from[h] = f, bytes[h] = uint32_t(l - f);
                        if (f > s || l < e) {  // odd elements at the row's ends
                            Y* const at = reinterpret_cast<Y*>(to + (lane + 32 * h) * pitch + (s - low));
                            for (uintptr_t x = s; x < e; x += ES) {
                                if (x >= f && x < l) x = l;
                                if (x < e && VCE_BOUNDS(lane + 32 * h < tile.count && x - low + ES <= uintptr_t(pitch), a.dev_status))
                                    at[(x - s) / ES] = *reinterpret_cast<const Y*>(x);
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a later round's copies
                        }
                    }
                    if (lane == 0 && tile.adapter >= 0) {
                        b_bytes = uint32_t((ve - v) * a.rank * 2);
                        if (first) t_bytes = uint32_t(tile.count * a.rank * 4);
                    }
                }
                if (lane == 0) ring.what[stage] = make_int4(end ? -1 : 0, v, ve - v, first);
                if (first) {
                    TileInfo<Y>& info = infos[stage];
                    if (lane == 0) info.adapter = tile.adapter, info.count = tile.count, info.scale = scale;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (row[h] != 0) {
                            info.out[lane + 32 * h] = static_cast<Y*>(a.out) + token[h] * a.out_stride;
                            info.off[lane + 32 * h] = int(row[h] & 15);
                        }
                    fresh = false;
                }
                mbar_arrive_expect_tx(&ring.full[stage], bytes[0] + bytes[1] + b_bytes + t_bytes);
                auto copy = [&](uint8_t* dst, const void* src, uint32_t n) {
                    if (VCE_BOUNDS(aligned16(src) && aligned16(dst) && n % 16 == 0 && dst + n <= to + a.stage_bytes, a.dev_status))
                        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                         smem_u32(dst)),
                                     "l"(src), "r"(n), "r"(smem_u32(&ring.full[stage]))
                                     : "memory");
                };
                if (t_bytes) copy(to + a.y_bytes + a.b_bytes, a.t + int64_t(tile.start) * a.rank, t_bytes);
                if (b_bytes) copy(to + a.y_bytes, a.b + (int64_t(tile.adapter) * a.vocab + v) * a.rank, b_bytes);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (bytes[h]) {
                        const uintptr_t low = (row[h] + int64_t(v) * ES) & ~uintptr_t(15);
                        copy(to + (lane + 32 * h) * pitch + (from[h] - low), reinterpret_cast<const void*>(from[h]), bytes[h]);
                    }
                ++issued;
                if (++stage == a.stages) stage = 0, parity ^= 1;
            }
            if (end || !ok) break;
            if (other) enter(next_tile);
            unit = next;
        }
        if (!ok) {  // copies on their way still write to shared memory
            if (lane == 0) report(a.dev_status, VCE_DEVSTATUS_TIMEOUT);
            for (int i = max(0, issued - a.stages); i < issued; ++i) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(&ring.full[i % a.stages], (i / a.stages) & 1) && globaltimer() - t0 < kDrainTimeoutNs) {}
            }
        }
        __syncthreads();
        return;
    }
    uint32_t parity = 0;
    int adapter = -1, pitch = 0, p0 = 0, part = 0, parts = 1, count = 0;
    // column 2 q + e of product j is token p0 + 8 j + 2 q + e: its row in a stage, and in memory
    int place[2][2];
    Y* to[2][2];
    uint32_t t[2][TERMS][KS][2];  // operands
    const int b_row = a.rank * 2;
    // The products of 32 logits, whose rows of B start at ``b``; EVERY: all 16 KS ranks are there.
    auto multiply = [&](float (&c)[2][2][4], const uint8_t* b, auto every) {
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
            const int r = rank_of<KS>(s, q);
            uint32_t w[2][2][4];  // product, row, words: row g of product i is logit 4 g + 2 i, row g + 8 the next
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* const from = b + (2 * i + h) * b_row + r * 2;
                    if constexpr (KS == 1) {
                        const uint2 x = decltype(every)::value || r < a.rank ? *reinterpret_cast<const uint2*>(from) : make_uint2(0, 0);
                        w[i][h][0] = x.x, w[i][h][1] = x.y;
                    } else {
                        const uint4 x = decltype(every)::value || r < a.rank ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
                        w[i][h][0] = x.x, w[i][h][1] = x.y, w[i][h][2] = x.z, w[i][h][3] = x.w;
                    }
                }
            auto step = [&](int j) {
#pragma unroll
                for (int e = 0; e < (KS == 1 ? 1 : 2); ++e)
#pragma unroll
                    for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t x[4] = {w[i][0][2 * e], w[i][1][2 * e], w[i][0][2 * e + 1], w[i][1][2 * e + 1]};
                            if (s + e == 0 && k == TERMS - 1) mma_first(c[i][j], x, t[j][k][s + e][0], t[j][k][s + e][1]);
                            else mma(c[i][j], x, t[j][k][s + e][0], t[j][k][s + e][1]);
                        }
            };
            step(0);
            if (count > 8) step(1);
        }
    };
    for (;;) {
        ok = mbar_wait(&ring.full[stage], parity, &ring.abort, kPipeTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int4 what = ring.what[stage];
        if (what.x < 0) break;
        uint8_t* const y = smem + size_t(stage) * a.stage_bytes;
        if (what.w) {
            const TileInfo<Y>& info = infos[stage];
            adapter = info.adapter;
            const int all = info.count, across_log2 = max(class_of(all) - 1, 0);  // warps across the tokens
            pitch = a.block[class_of(all)] * ES + 32;
            p0 = (warp & ((1 << across_log2) - 1)) * 16, part = warp >> across_log2, parts = kMulWarps >> across_log2;
            count = min(16, all - p0);  // of this warp's tokens; none if not positive
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = 8 * j + 2 * q + e;
                    to[j][e] = nullptr, place[j][e] = 0;
                    if (p < count) to[j][e] = info.out[p0 + p], place[j][e] = (p0 + p) * pitch + info.off[p0 + p];
                }
            if (adapter >= 0) {
                const float scale = info.scale;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        const int p = 8 * j + g, r = rank_of<KS>(s, q);
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (p < count && r < a.rank)
                            x = *reinterpret_cast<const float4*>(y + a.y_bytes + a.b_bytes + ((p0 + p) * a.rank + r) * 4);
                        uint32_t w[2][TERMS];
                        split2<TERMS>(x.x * scale, x.y * scale, w[0]);
                        split2<TERMS>(x.z * scale, x.w * scale, w[1]);
#pragma unroll
                        for (int k = 0; k < TERMS; ++k) t[j][k][s][0] = w[0][k], t[j][k][s][1] = w[1][k];
                    }
            }
        }
        const int here = what.z;
#pragma unroll 1
        for (int vc = part * 32; vc < here && count > 0; vc += parts * 32) {
            uint8_t* const yc = y + vc * ES;
            const int64_t vo = what.y + vc;
            if (!VCE_BOUNDS(vo >= 0 && what.y + here <= a.vocab && (vc + 32) * ES + 16 <= pitch &&
                                (vc + 32) * b_row <= a.b_bytes && (p0 + count) * pitch <= a.y_bytes,
                            a.dev_status))
                break;
            if (adapter >= 0) {
                float c[2][2][4];
                const uint8_t* const b = y + a.y_bytes + (vc + 4 * g) * b_row;
                if (a.rank == KS * 16) multiply(c, b, std::true_type{});
                else multiply(c, b, std::false_type{});
                const int left = here - vc - 4 * g;  // of this lane's four logits
                const bool whole = vc + 32 <= here;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (8 * j >= count) break;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (to[j][e] == nullptr) continue;
                        const float sum[4] = {c[0][j][e], c[0][j][2 + e], c[1][j][e], c[1][j][2 + e]};
                        Y* const at = reinterpret_cast<Y*>(yc + place[j][e]) + 4 * g;
                        if constexpr (VEC) {
                            float x[4];
                            load4(x, at);  // (past the end: of the stage, not used)
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[i] += sum[i];
                            Y* const out = to[j][e] + vo + 4 * g;
                            if (whole || left >= 4) {
                                store4(out, x);
                            } else {
#pragma unroll
                                for (int i = 0; i < 3; ++i)
                                    if (i < left) put(out + i, x[i]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (whole || i < left) put(at + i, to_float(at[i]) + sum[i]);
                        }
                    }
                }
            }
            if (!VEC || adapter < 0) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (8 * j >= count) break;
#pragma unroll
                    for (int p = 0; p < 8; ++p) {  // token 8 j + p is lane p / 2's, its (p % 2)-th
                        if (8 * j + p >= count) break;
                        const int where = __shfl_sync(0xffffffffu, place[j][p & 1], p >> 1);
                        Y* const out = reinterpret_cast<Y*>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to[j][p & 1]), p >> 1));
                        if (vc + lane < here) out[vo + lane] = (reinterpret_cast<const Y*>(yc + where))[lane];
                    }
                }
            }
        }
        if constexpr (!VEC) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.empty[stage]);
        if (++stage == a.stages) stage = 0, parity ^= 1;
    }
    __syncthreads();
}

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

// Up to kVBlock neighbouring logits of a row that starts anywhere, held by a warp: whole vectors by the address that is
// written, and an element per lane of what comes before and behind them.
template <typename Y>
struct SomeRow {
    static constexpr int VE = 16 / int(sizeof(Y)), kChunks = kVBlock / VE / 32;
    uint32_t v[kChunks][4];
    Y single;

    // Elements of a row before its first 16-byte boundary.
    __device__ __forceinline__ static int before(const Y* p) {
        return int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / sizeof(Y));
    }
    // This lane's single element of ``n``, or -1.
    __device__ __forceinline__ static int one(int head, int n) {
        const int lane = threadIdx.x & 31, i = lane < VE ? lane : ((n - head) & ~(VE - 1)) + head + lane - VE;
        return i < (lane < VE ? head : n) ? i : -1;
    }
    __device__ __forceinline__ static uint32_t word(const float* p) { return __float_as_uint(*p); }
    __device__ __forceinline__ static uint32_t word(const __nv_bfloat16* p) {
        return uint32_t(__bfloat16_as_ushort(p[0])) | uint32_t(__bfloat16_as_ushort(p[1])) << 16;
    }
    // ``head`` (at most n) elements lie before out's vectors; ``alike``: and before y's.
    __device__ __forceinline__ void load(const Y* y, int head, bool alike, int n) {
        const int lane = threadIdx.x & 31, whole = (n - head) / VE;
        const Y* const at = y + head + lane * VE;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (lane + 32 * k < whole) {
                const Y* const x = at + 32 * VE * k;
                if (alike) w = *reinterpret_cast<const uint4*>(x);
                else w = make_uint4(word(x), word(x + VE / 4), word(x + VE / 2), word(x + 3 * VE / 4));
            }
            v[k][0] = w.x, v[k][1] = w.y, v[k][2] = w.z, v[k][3] = w.w;
        }
        const int i = one(head, n);
        single = Y(0.f);
        if (i >= 0) single = y[i];
    }
    __device__ __forceinline__ void copy(Y* out, int head, int n) const {
        const int lane = threadIdx.x & 31, whole = (n - head) / VE;
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
            if (lane + 32 * k < whole)
                *reinterpret_cast<uint4*>(out + head + (lane + 32 * k) * VE) = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        const int i = one(head, n);
        if (i >= 0) out[i] = single;
    }
    // ``sums``: of logit i at i + i / 8.
    __device__ __forceinline__ void add(Y* out, int head, int n, const float* sums) {
        const int lane = threadIdx.x & 31, whole = (n - head) / VE;
        auto sum = [&](int i) { return sums[i + (i >> 3)]; };
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            if (lane + 32 * k >= whole) continue;
            const int i0 = head + (lane + 32 * k) * VE;
            if constexpr (VE == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[k][i] = __float_as_uint(__uint_as_float(v[k][i]) + sum(i0 + i));
            } else {
                const float* const at = sums + 9 * lane + head;
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = at[i + (head + i >= 8)];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[k][i] = Eight<__nv_bfloat16>::sum(v[k][i], x[2 * i], x[2 * i + 1]);
            }
            *reinterpret_cast<uint4*>(out + i0) = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        }
        const int i = one(head, n);
        if (i >= 0) put(out + i, to_float(single) + sum(i));
    }
};

// Operands of B for logits v0 .. v0 + 31 of adapter_expand_many.
template <int KS>
__device__ __forceinline__ void load_b(uint32_t (&b)[4][KS][2], const ExpandArgs& a, int adapter, int v0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int v = v0 + 8 * (g >> 1) + 2 * j + (g & 1);
        const __nv_bfloat16* const at = a.b + (int64_t(adapter) * a.vocab + v) * a.rank;
        if constexpr (KS == 1) {
            uint2 w = make_uint2(0, 0);
            if (v < a.vocab && 4 * q < a.rank && VCE_BOUNDS((reinterpret_cast<uintptr_t>(at) & 7) == 0, a.dev_status))
                w = __ldg(reinterpret_cast<const uint2*>(at + 4 * q));
            b[j][0][0] = w.x, b[j][0][1] = w.y;
        } else {
#pragma unroll
            for (int s = 0; s < KS; s += 2) {
                const int r = rank_of<KS>(s, q);
                uint4 w = make_uint4(0, 0, 0, 0);
                if (v < a.vocab && r < a.rank && VCE_BOUNDS(aligned16(at + r), a.dev_status))
                    w = __ldg(reinterpret_cast<const uint4*>(at + r));
                b[j][s][0] = w.x, b[j][s][1] = w.y, b[j][s + 1][0] = w.z, b[j][s + 1][1] = w.w;
            }
        }
    }
}

// Many tokens to an adapter, large ranks, or little work.  Tokens are the rows of the products (16)
// and logits the columns (8): column 2 q + e of product j is logit 8 q + 2 j + e of the warp's 32, so that
// a lane ends up with eight neighbours of a row.  A warp loads B's operands once for all tokens of a tile, and
// the next rows of y while it multiplies.
//
// Units are blocks of kVBlock logits of a tile, tiles of the same logits next to each other: blocks that
// work at the same time read the same part of B.  Where tiles are few a block stays with its tile; where they hold few
// tokens a unit has several blocks of logits, so that the tile's operands of t are put together less often.
//
// Rows that start anywhere (VEC false): the products of 16 tokens go through shared memory, from which each warp
// adds them to two rows, in the vectors that lie at 16-byte boundaries of the row; what is left at the ends of
// its kVBlock logits takes an element per lane.
//
// 2048 tokens with 6 adapters of rank 64, 128256 BF16 logits: 263 us (4.3 TB/s; under the profiler).  It is
// bound by what 16 warps per SM keep on its way between their instructions.  More rows on their way help small
// ranks (512 x 128256, rank 16, BF16: 86 -> 76 us in all) and cost as much with large ones (2048 tokens of rank
// 64: 291 -> 318).  Rows of 128257 logits take 455 us in all (element by element through the warps' own shared memory 660).
//
// All three kernels in us, this form / the other one: 512 x 128256, rank 16, 16 tokens per adapter
// 110 / 96 (BF16), 137 / 128 (FP32); 32 tokens 80 / 103 and 117 / 163; hence kMany.  16 tokens with 16 adapters, rank 16,
// BF16: 8000 logits 13 / 15, 32000 17 / 21, 128256 29 / 27; 32 with 32: 15 / 17, 21 / 22, 52 / 41; hence kShort.
// Off 16-byte boundaries 257 with 20, 32001 logits 45 / 37; 16 with 16 19 / 21; hence kShortAny.
// 1024 with 64, 128256 FP32: rank 32 398 / 346, rank 64 504 / 451, in BF16 319 / 245 and 368 / 680.
template <typename Y, int KS, bool VEC>
__global__ void __launch_bounds__(kThreads, KS <= 4 ? 2 : 1) adapter_expand_many(const __grid_constant__ ExpandArgs a) {
    constexpr int TERMS = sizeof(Y) == 2 ? 2 : 3;
    constexpr int kAhead = KS > 2 || !VEC ? 1 : sizeof(Y) == 2 ? 4 : 3;  // groups of 16 rows on their way
    constexpr int kSlots = kAhead < kMTiles ? kAhead + 1 : kMTiles;
    extern __shared__ __align__(16) uint4 frag[];  // [TERMS][kMTiles][KS][32]: operands of t; then each warp's products
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    cudaGridDependencySynchronize();
    const int vblocks = (a.vocab + kVBlock - 1) / kVBlock, tiles = a.plan->n_all;
    const int run = int64_t(tiles) * 32 <= a.n ? 1 : int(max(int64_t(1), min(int64_t(8), int64_t(tiles) * vblocks / (3 * int64_t(gridDim.x)))));
    const int64_t units = int64_t(tiles) * ((vblocks + run - 1) / run);
    const int step = tiles * 4 <= int(gridDim.x) ? int(gridDim.x) / max(tiles, 1) * tiles : int(gridDim.x);
    if (int(blockIdx.x) >= step) return;
    int id = -1;
    Tile tile{};
    int token[kMTiles][2];  // VEC
    struct Place {  // of a token's row
        const Y* y;
        Y* out;
        int head, alike;  // as of SomeRow
    };
    __shared__ __align__(16) char place_mem[VEC ? 16 : kTile * sizeof(Place)];
    Place* const place = reinterpret_cast<Place*>(place_mem);
    float* const cells = reinterpret_cast<float*>(frag + TERMS * kMTiles * KS * 32);  // two of them, in turn
    int turn = 0;
    for (int64_t unit = blockIdx.x; unit < units; unit += step) {
        const int now = int(unit % tiles), vb0 = int(unit / tiles) * run;
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
                        if (p < tile.count && r < a.rank && VCE_BOUNDS(tile.start + p < a.n, a.dev_status))
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
            if constexpr (!VEC)
                if (tid < tile.count) {
                    const int64_t n = token_at(a.perm, tile.start + tid, a.n, a.dev_status);
                    const Y* const y = static_cast<const Y*>(a.y) + n * a.y_stride;
                    Y* const out = static_cast<Y*>(a.out) + n * a.out_stride;
                    place[tid] = {y, out, SomeRow<Y>::before(out), SomeRow<Y>::before(y) == SomeRow<Y>::before(out)};
                }
#pragma unroll
            for (int m = 0; m < (VEC ? kMTiles : 0); ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = m * 16 + h * 8 + g;
                    token[m][h] = p < tile.count ? token_at(a.perm, tile.start + p, a.n, a.dev_status) : -1;
                }
            __syncthreads();
        }
        // Tokens without an adapter: y as it is, every bit (the sum with +0 would make +0 of -0).
        if constexpr (VEC) {
            if (tile.adapter < 0) {
                for (int vb = vb0; vb < min(vb0 + run, vblocks); ++vb) {
                    const int v = vb * kVBlock + warp * kVWarp + 8 * q, left = a.vocab - v;
                    if (left <= 0) continue;
                    Eight<Y> e[kMTiles][2];
#pragma unroll
                    for (int m = 0; m < kMTiles; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            e[m][h].clear();  // (what a load may leave undefined is spilled, in the loop below too: 1182 us instead of 446)
                            if (token[m][h] < 0) continue;
                            const Y* const p = static_cast<const Y*>(a.y) + token[m][h] * a.y_stride + v;
                            if (!VCE_BOUNDS(aligned16(p), a.dev_status)) continue;
                            if (left >= 8) e[m][h].load(p);
                            else e[m][h].load_some(p, left);
                        }
#pragma unroll
                    for (int m = 0; m < kMTiles; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (token[m][h] < 0) continue;
                            Y* const p = static_cast<Y*>(a.out) + token[m][h] * a.out_stride + v;
                            if (!VCE_BOUNDS(aligned16(p), a.dev_status)) continue;
                            if (left >= 8) e[m][h].store(p);
                            else e[m][h].store_some(p, left);
                        }
                }
                continue;
            }
        }
        for (int vb = vb0; vb < min(vb0 + run, vblocks); ++vb) {
            const int v0 = vb * kVBlock + warp * kVWarp;
            if (VEC && v0 >= a.vocab) continue;
            uint32_t b[4][KS][2];
            // (a condition that the compiler does not see through: without it the loads of y wait, 512 x 128256, rank 16,
            // BF16, 92 us in all instead of 83)
            int adapter = tile.adapter;
            asm volatile("" : "+r"(adapter));
            if (adapter >= 0) load_b<KS>(b, a, adapter, v0);
            auto multiply = [&](float (&c)[4][4], int m) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int k = TERMS - 1; k >= 0; --k) {
                        const uint4 f = frag[((k * kMTiles + m) * KS + s) * 32 + lane];
                        const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (s == 0 && k == TERMS - 1) mma_first(c[j], w, b[j][s][0], b[j][s][1]);
                            else mma(c[j], w, b[j][s][0], b[j][s][1]);
                        }
                    }
            };
            if constexpr (VEC) {
                const int v = v0 + 8 * q, left = a.vocab - v;  // this lane's eight logits
                const bool whole = left >= 8;
                auto fetch = [&](Eight<Y>& e, int n) {
                    e.clear();  // (a load that may not be made would wait for what the registers held)
                    if (n < 0 || left <= 0) return;
                    const Y* const p = static_cast<const Y*>(a.y) + n * a.y_stride + v;
                    if (!VCE_BOUNDS(aligned16(p) && v >= 0, a.dev_status)) return;
                    if (whole) e.load(p);
                    else e.load_some(p, left);
                };
                Eight<Y> e[kSlots][2];
#pragma unroll
                for (int m = 0; m < kAhead; ++m) {
                    fetch(e[m][0], token[m][0]);
                    fetch(e[m][1], token[m][1]);
                }
#pragma unroll
                for (int m = 0; m < kMTiles; ++m) {
                    if (m * 16 >= tile.count) break;
                    if (m + kAhead < kMTiles) {  // before the products: a load behind their stores would wait for them
                        const int next = m + kAhead < kMTiles ? m + kAhead : 0;
                        fetch(e[next % kSlots][0], token[next][0]);
                        fetch(e[next % kSlots][1], token[next][1]);
                    }
                    float c[4][4];
                    multiply(c, m);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        Eight<Y>& x = e[m % kSlots][h];
                        const int n = token[m][h];
                        if (n >= 0 && left > 0) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) x.add(j, c[j][2 * h], c[j][2 * h + 1]);
                            Y* const p = static_cast<Y*>(a.out) + n * a.out_stride + v;
                            if (!VCE_BOUNDS(aligned16(p), a.dev_status)) continue;
                            if (whole) x.store(p);
                            else x.store_some(p, left);
                        }
                    }
                }
            } else {
                const int base = vb * kVBlock, here = min(kVBlock, a.vocab - base);
                auto fetch = [&](SomeRow<Y>(&x)[2], int m) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int p = m * 16 + 2 * warp + r;
                        const Place at = place[p];
                        const bool is = p < tile.count;
                        x[r].load(at.y + base, is ? min(at.head, here) : 0, at.alike, is ? here : 0);
                    }
                };
                if (tile.adapter < 0) {  // (not before the loop, as above: 600 x 32001 FP32 57 us instead of 51)
                    SomeRow<Y> e[kMTiles][2];
#pragma unroll
                    for (int m = 0; m < kMTiles; ++m) fetch(e[m], m);
#pragma unroll
                    for (int m = 0; m < kMTiles; ++m)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int p = m * 16 + 2 * warp + r;
                            if (p < tile.count) e[m][r].copy(place[p].out + base, min(place[p].head, here), here);
                        }
                    continue;
                }
                SomeRow<Y> e[kSlots][2];
#pragma unroll
                for (int m = 0; m < kAhead; ++m) fetch(e[m], m);
#pragma unroll
                for (int m = 0; m < kMTiles; ++m) {
                    if (m * 16 >= tile.count) break;
                    if (m + kAhead < kMTiles) fetch(e[(m + kAhead) % kSlots], m + kAhead);
                    float c[4][4];
                    multiply(c, m);
                    float* const cell = cells + turn * (16 * kCellPitch);
                    turn ^= 1;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float* const at = cell + (h * 8 + g) * kCellPitch + 9 * (4 * warp + q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) at[2 * j] = c[j][2 * h], at[2 * j + 1] = c[j][2 * h + 1];
                    }
                    __syncthreads();  // (the next one comes before this cell's next turn)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int p = m * 16 + 2 * warp + r;
                        if (p < tile.count)
                            e[m % kSlots][r].add(place[p].out + base, min(place[p].head, here), here, cell + (2 * warp + r) * kCellPitch);
                    }
                }
            }
        }
    }
}

template <typename Y, bool VEC>
auto few_kernel(int ks) {
    return ks == 1 ? adapter_expand_few<Y, 1, VEC> : adapter_expand_few<Y, 2, VEC>;
}

template <typename Y, bool VEC>
auto many_kernel(int ks) {
    return ks == 1 ? adapter_expand_many<Y, 1, VEC> : ks == 2 ? adapter_expand_many<Y, 2, VEC>
                                                  : ks == 4 ? adapter_expand_many<Y, 4, VEC> : adapter_expand_many<Y, 8, VEC>;
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
    const PlanArgs pa{index, int(n), int(adapters), !in_place, int(most_tiles(n, adapters)), w.plan, w.tiles, w.perm, dev_status};
    const bool self = n <= kSelf;
    if (!self) {
        count_launch();
        adapter_plan<<<1, kPlanThreads, 0, s>>>(pa);
        if (cudaGetLastError() != cudaSuccess) return VCE_ERR_CUDA;
    }
    // by the hidden dimension alone: a token's sums are divided in the same way in every batch
    const int slices = hidden > 1024 ? 8 : hidden > 512 ? 4 : hidden > 256 ? 2 : 1;

    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(slices);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;

    const ShrinkArgs sa{pa, slices, x, x_stride, static_cast<const __nv_bfloat16*>(a), int(hidden), rank, int(n), w.plan, w.tiles,
                        w.perm, w.t, dev_status};
    auto shrink = x_dtype == VCE_BF16 ? (self ? adapter_shrink<__nv_bfloat16, true> : adapter_shrink<__nv_bfloat16, false>)
                                      : (self ? adapter_shrink<float, true> : adapter_shrink<float, false>);
    const size_t shrink_smem = size_t(kWarps) * kTile * kRankBlock * 4;
    const int ks = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
    const int es = y_dtype == VCE_BF16 ? 2 : 4;
    const bool vectors = reinterpret_cast<uintptr_t>(y) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                         (n == 1 || (y_stride * es % 16 == 0 && out_stride * es % 16 == 0));
    const int64_t used = std::min(n, adapters), vblocks = (vocab + kVBlock - 1) / kVBlock;
    const int many_blocks = dev.num_sms * (ks <= 4 ? 2 : 1);
    const bool many = ks > 2 || n >= kMany * used || (used + n / kTile) * vblocks <= (vectors ? kShort : kShortAny) * many_blocks;
    const size_t many_smem = size_t(y_dtype == VCE_BF16 ? 2 : 3) * kMTiles * ks * 32 * sizeof(uint4) +
                             (vectors ? 0 : size_t(2) * 16 * kCellPitch * sizeof(float));
    auto expand = many ? y_dtype == VCE_BF16
                             ? (vectors ? many_kernel<__nv_bfloat16, true>(ks) : many_kernel<__nv_bfloat16, false>(ks))
                             : (vectors ? many_kernel<float, true>(ks) : many_kernel<float, false>(ks))
                  : y_dtype == VCE_BF16 ? (vectors ? few_kernel<__nv_bfloat16, true>(ks) : few_kernel<__nv_bfloat16, false>(ks))
                                        : (vectors ? few_kernel<float, true>(ks) : few_kernel<float, false>(ks));
    ExpandArgs ea{static_cast<const __nv_bfloat16*>(b), scale, w.t, y, out, y_stride, out_stride, int(n), int(vocab), rank, 0, 0, 0, 0,
                  {}, w.plan, w.tiles, w.perm, dev_status};
    if (!many) {  // three stages at least
        const int t_bytes = kTile * rank * 4, b_most = std::min(kStageB, kRingBytes / 3 - (kStageRows + kTile * 32) - t_bytes);
        for (int rows : {4, 16, 32, 64}) {
            int& block = ea.block[class_of(rows)];
            block = std::min({kMaxBlock, kStageRows / (rows * es), b_most / (rank * 2)}) / 32 * 32;
            ea.y_bytes = std::max(ea.y_bytes, rows * (block * es + 32));
            ea.b_bytes = std::max(ea.b_bytes, block * rank * 2);
        }
        ea.stage_bytes = ea.y_bytes + ea.b_bytes + t_bytes;  // multiples of 64 all
        ea.stages = std::min(kMaxStages, kRingBytes / ea.stage_bytes);
    }
    static std::mutex mu;
    static bool ready[64], ready_expand[64][2][2][2][4];
    {
        std::lock_guard<std::mutex> lock(mu);
        bool& done = ready_expand[dev.ordinal][many][y_dtype == VCE_BF16][vectors][ks == 8 ? 3 : ks / 2];
        if (!done && cudaFuncSetAttribute(expand, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          int(many ? many_smem : size_t(kRingBytes))) != cudaSuccess)
            return VCE_ERR_CUDA;
        done = true;
        if (!ready[dev.ordinal]) {
            for (auto k : {adapter_shrink<__nv_bfloat16, true>, adapter_shrink<__nv_bfloat16, false>, adapter_shrink<float, true>,
                           adapter_shrink<float, false>})
                if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shrink_smem)) != cudaSuccess)
                    return VCE_ERR_CUDA;
            ready[dev.ordinal] = true;
        }
    }
    cfg.gridDim = dim3(unsigned(used + n / kTile) * slices, unsigned((rank + kRankBlock - 1) / kRankBlock));
    cfg.dynamicSmemBytes = shrink_smem;
    if (self) cfg.attrs = attr + 1;  // the first kernel of the call: what runs before it is not ours
    cfg.numAttrs = self ? 1 : 2;
    count_launch();
    if (cudaLaunchKernelEx(&cfg, shrink, sa) != cudaSuccess) return VCE_ERR_CUDA;
    cfg.attrs = attr;

    if (many) {
        cfg.gridDim = dim3(unsigned(many_blocks));
        cfg.dynamicSmemBytes = many_smem;
        cfg.numAttrs = 1;
        count_launch();
        return cudaLaunchKernelEx(&cfg, expand, ea) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
    }
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(most_tiles(n, adapters) * ((vocab + kRun - 1) / kRun), int64_t(dev.num_sms))));
    cfg.blockDim = dim3(kMulWarps * 32 + 32);
    cfg.dynamicSmemBytes = size_t(ea.stages) * ea.stage_bytes;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, expand, ea) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
