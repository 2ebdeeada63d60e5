// Product of microscaled matrices: logits[n, v] = sum_k x[n, k] w[v, k], x in E4M3 and
// the classifier w in E2M1, each with one power-of-two scale per 32 values of k.
//
// tcgen05.mma.kind::mxf8f6f4 with block scales multiplies such operands as they are:
// products of codes are exact, the two scales of a block of 32 are applied inside the
// tensor core and sums are FP32.  Tokens are the M operand (128 of them, one per
// tensor-memory lane) and the classifier's rows the N operand, for few tokens too: an
// instruction with N = 16 tokens over 128 classifier rows costs nearly as much as one
// with N = 128, and the classifier is what has to be fed through (8 tokens x 4096 x
// 128256: 105 us that way round).
//
// 4-bit values travel packed (two per byte) from HBM.  The tensor core wants them in
// shared memory as 16-byte pieces of 16 values, 8 bytes of codes and 8 of padding, and
// a tensor map of type 16U4_ALIGN16B makes the copy engine spread them so (counting the
// packed bytes on the barrier).  Converter warps in its place took as many cycles of
// shared memory as feeding the tensor core (83 us at 8 tokens, 1005 us at 2048).
//
// Times at 4096 x 128256 with BF16 logits: 8 tokens 53 us, bound by memory (281 MB, 0.79 of
// the copy rate; the rest is the start of the pipeline and a last round that is half full);
// 2048 tokens (in CTA pairs) 588 us, 3.7 PFLOP/s, bound by the tensor core, and by the power
// limit where calls follow one another for long.
//
// Roles: warp 0 copies both operands and their scales (TMA), warp 1 issues the MMAs, warps
// 4 to 11 drain accumulators.  One ring of 128 columns per stage.  Every wait is
// bounded, as in lce_tc.cu.

#include "head_internal.cuh"
#include "mx_format.cuh"
#include "mx_plan.h"
#include "sm100_ptx.cuh"

#include <cudaTypedefs.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kTokens = mx::kLinearTokens;      // per tile
constexpr int kK = 128;                         // columns per stage: one 128-byte swizzle row
constexpr int kRows = mx::kLinearRows;          // of the classifier per tile; the last tiles may have half
constexpr uint32_t kWBytes = kRows * kK;        // as the tensor core reads them: half is padding
constexpr int kFirstEpilogue = 4;               // warp; a multiple of 4, as lane quadrants go by warp % 4
constexpr int kEpilogueWarps = 8;               // four per 128 columns
constexpr int kThreads = (kFirstEpilogue + kEpilogueWarps) * 32;
constexpr int kTurnCols = 16;                   // columns an epilogue warp turns at a time
constexpr uint32_t kTurnBytes = 32 * (kTurnCols + 1) * 4;  // and its scratch
// Tensor memory: two accumulators of 256 columns that share 16 (0-255 and 240-495), x's
// scales (4 columns) and w's (8) behind them.  A tile's shared columns are drained first,
// then the next tile's MMAs may start.
constexpr uint32_t kAccStep = 240, kScaleCol = 496, kTmemCols = 512;

// XR: rows of x a stage has room for.  Fewer than a tile's 128 serve fewer tokens: the
// tensor core then reads its other rows from w's tile behind them, whatever that means as
// E4M3, into accumulator rows that nobody stores.
template <int XR>
struct Cfg {
    static constexpr uint32_t kXBytes = XR * kK;
    static constexpr uint32_t kStage = kXBytes + kWBytes;
    static constexpr uint32_t kScales = 3 * mx::kTileBytes;  // x, w, w
    static constexpr int kStages = XR == 128 ? 4 : 5;
    static constexpr size_t kSmem = size_t(kStages) * (kStage + kScales) + kEpilogueWarps * kTurnBytes + 1024 + 512;
    static_assert((kTokens - XR) * kK <= int(kWBytes) / 2 && kSmem <= 232448, "shared memory");
};

struct LinearArgs {
    int64_t n, v;
    int k_tiles;           // 128-column tiles
    int tiles_v, tiles_n;  // tiles of classifier rows and of tokens
    int whole_v;           // the first so many tiles have 256 rows, the others 128
    int64_t w_scale_rows;  // 128-row tiles of w's scales
    const uint8_t *w_scales, *x_scales;
    void* out;
    int64_t out_stride;
    int wide;              // every 32 columns of a row start 16-byte (1) or 32-byte (2) aligned
    int* dev_status;
    uint64_t timeout_ns;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Matrix descriptors as (low, high) words: everything but the start address (>> 4, in
// the low word) is the same for all of a kind, so that the issuing thread, whose
// instructions one by one are what a short stage waits for, only adds to the low word.
//   operand tiles: 128-byte swizzle, 8-row atoms 1024 bytes apart (see sm100_ptx.cuh)
//   scale tiles: 32 rows of 16 bytes without swizzle, 8-row groups 128 bytes apart
constexpr uint32_t kTileHigh = (1024 >> 4) | 1u << 14 | 2u << 29, kTileLow = (16 >> 4) << 16;
constexpr uint32_t kScaleHigh = (128 >> 4) | 1u << 14, kScaleLow = (128 >> 4) << 16;

// A 512-byte scale tile into four tensor-memory columns (rows 32 j .. 32 j + 31 in
// column j, a byte per 32 columns of k), repeated in all four lane quadrants.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t low) {
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\ttcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(low), "n"(kScaleHigh)
        : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: A E4M3 (0) at bit 7, B E2M1 (5) at bit 10,
// N >> 3 at bit 17, E8M0 scales (bit 23), M >> 4 at bit 24; the byte of the scale
// columns that holds this k step at bits 29 (A) and 4 (B).
constexpr uint32_t kScaleIdStep = 1u << 29 | 1u << 4;  // the next k step's scales
__device__ constexpr uint32_t idesc_mx(int n, int k_step) {
    return (5u << 10) | (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(kTokens >> 4) << 24) |
           (uint32_t(k_step) << 29) | (uint32_t(k_step) << 4);
}

__device__ __forceinline__ void umma_mx(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kTileHigh)
        : "memory");
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// A whole warp's wait: every lane polls.  (A branch that only one lane takes costs its
// warp about as much as the handover itself: a round trip between two warps measured 285
// clocks with all lanes polling, 472 with one.)
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
    return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, abort, timeout_ns));
}

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 32 consecutive logits of one token as words.  Rows that start 32-byte aligned are stored by
// 32 bytes, whole sectors of L2: the stores of 16 bytes, two requests per sector, bound the
// kernel where tiles are short (2048 x 1024 x 128256 BF16: 315 us by 16 bytes, 219 by 32).
__device__ __forceinline__ void store_words(void* p, const uint32_t* u, int words, bool sectors) {
    if (sectors) {
#pragma unroll
        for (int i = 0; i < words; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<uint32_t*>(p) + i),
                         "r"(u[i]), "r"(u[i + 1]), "r"(u[i + 2]), "r"(u[i + 3]), "r"(u[i + 4]), "r"(u[i + 5]),
                         "r"(u[i + 6]), "r"(u[i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < words; i += 4)
            *reinterpret_cast<uint4*>(static_cast<uint32_t*>(p) + i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
    }
}
__device__ __forceinline__ uint32_t logit_pair(uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store_row32(float* p, const uint32_t (&r)[32], bool sectors) {
    store_words(p, r, 32, sectors);
}
__device__ __forceinline__ void store_row32(__nv_bfloat16* p, const uint32_t (&r)[32], bool sectors) {
    uint32_t u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = logit_pair(r[2 * i], r[2 * i + 1]);
    store_words(p, u, 16, sectors);
}

// The first ``left`` of 32 consecutive logits of ``live`` tokens (one per lane) in rows at any
// offset from ``out`` on: turned through shared memory, so that half a warp stores 16
// neighbouring logits of one token.  (BF16 logits two to a word, with the odd rows' words put
// together from neighbours, took 64 us where this takes 45: 1024 x 512 x 32001.)
template <typename Out>
__device__ __forceinline__ void store_turned(Out* out, int64_t stride, const uint32_t (&r)[32], int live, int left,
                                             float* mine) {
    const int lane = threadIdx.x & 31, hl = lane & 15, hr = lane >> 4;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kTurnCols; ++j)
            mine[lane * (kTurnCols + 1) + j] = __uint_as_float(r[part * kTurnCols + j]);
        __syncwarp();
        const int c = part * kTurnCols + hl;
        if (c < left) {
            Out* p = out + int64_t(hr) * stride + c;
#pragma unroll 4
            for (int i = hr; i < live; i += 2, p += 2 * stride) store_logit(p, mine[i * (kTurnCols + 1) + hl]);
        }
    }
}

// Tile t of the launch: its classifier rows (first, width 256 or 128) and its tokens.
struct Tile {
    int64_t v0, n0;
    int width;
};
__device__ __forceinline__ Tile tile_at(const LinearArgs& a, int t) {
    const int tv = t / a.tiles_n, tn = t - tv * a.tiles_n;
    const bool whole = tv < a.whole_v;
    return {int64_t(whole ? tv : a.whole_v) * kRows + (whole ? 0 : int64_t(tv - a.whole_v) * 128), int64_t(tn) * kTokens,
            whole ? kRows : 128};
}

// An epilogue warp's part of a finished tile: one token per lane, from n0 on, and 128 logits
// from v0 on, below ``end``.  ``shared_drained`` is called (by one lane) when the columns
// that both accumulators have are out of tensor memory, if this warp has them.
template <typename Out, typename F>
__device__ __forceinline__ void store_tile(const LinearArgs& a, int64_t n0, int64_t v0, int64_t end, uint32_t accum,
                                           uint32_t acc, int q, int half, float* mine, F shared_drained) {
    const int lane = threadIdx.x & 31;
    const int live = int(a.n - n0 < 32 ? a.n - n0 : 32);  // tokens of this warp
    const int64_t right = a.v < end ? a.v : end;
    const int cols = int(right - v0 < 128 ? right - v0 : 128);
    const uint32_t taddr = accum + (uint32_t(q * 32) << 16) + half * 128;
    Out* out = static_cast<Out*>(a.out) + n0 * a.out_stride + v0;
    // the columns both accumulators have are the last of the first one's second half and
    // the first of the second one's first half
    const bool shares = half != int(acc);
    const bool work = live > 0 && cols > 0 && VCE_BOUNDS(n0 >= 0 && v0 >= 0, a.dev_status);
    if (shares && !work && lane == 0) shared_drained();
    if (work) {
        const int chunks = (cols + 31) / 32;
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
            const int c = (acc == 0 ? chunks - 1 - i : i) * 32;
            uint32_t r[32];
            tmem_ld32(taddr + c, r);
            tmem_ld_wait();
            if (shares && i == 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) shared_drained();
            }
            if (a.wide) {
                Out* row = out + int64_t(lane) * a.out_stride + c;
                if (lane < live) {
                    if (cols - c >= 32) {
                        store_row32(row, r, a.wide == 2);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < cols - c) store_logit(row + j, __uint_as_float(r[j]));
                    }
                }
            } else {
                store_turned(out + c, a.out_stride, r, live, min(32, cols - c), mine);
            }
        }
    }
}

template <int XR, typename Out>
__global__ void __launch_bounds__(kThreads, 1)
mx_linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                 const LinearArgs a) {
    using C = Cfg<XR>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* scales = smem + size_t(S) * C::kStage;  // stages of x, then w: multiples of 1024 bytes
    uint8_t* turn = scales + size_t(S) * C::kScales;
    uint64_t* full = reinterpret_cast<uint64_t*>(turn + kEpilogueWarps * kTurnBytes);
    uint64_t* empty = full + S;
    uint64_t* t_full = empty + S;    // a tile's MMAs are done
    uint64_t* t_empty = t_full + 2;  // its accumulator is drained
    uint64_t* shared_empty = t_empty + 2;  // the columns it shares with the other are
    uint64_t* drain = shared_empty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = a.tiles_v * a.tiles_n;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], kEpilogueWarps);
        }
        mbar_init(shared_empty, 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int no_abort = 0;

    if (warp == 0) {
        // ---------------- copies ----------------
        if (lane == 0) {
            tma_prefetch_desc(&tm_w);
            tma_prefetch_desc(&tm_x);
        }
        uint32_t s = 0, phase = 0, issued = 0, issued_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile tile = tile_at(a, t);
            const int64_t st = tile.v0 / 128;  // first scale tile of w
            const int wt = tile.width == kRows && st + 1 < a.w_scale_rows ? 2 : 1;
            const uint8_t* ws = a.w_scales + st * a.k_tiles * mx::kTileBytes;
            const uint8_t* xs = a.x_scales + tile.n0 / 128 * a.k_tiles * mx::kTileBytes;
            for (int k = 0; k < a.k_tiles; ++k) {
                ok = warp_wait(&empty[s], phase ^ 1u, abort_flag, a.timeout_ns);
                if (!ok) break;
                // past the last column and row the copies write zeros, which count as bytes; a
                // copy of w counts its packed bytes
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[s], C::kXBytes + tile.width * (kK / 2) + (1 + wt) * mx::kTileBytes);
                    const uint32_t sx = smem_u32(smem + size_t(s) * C::kStage);
                    const uint32_t sc = smem_u32(scales + size_t(s) * C::kScales);
                    if (VCE_BOUNDS(tile.v0 < a.v && tile.n0 < a.n && st + wt <= a.w_scale_rows, a.dev_status)) {
                        tma_load_2d(sx + C::kXBytes, &tm_w, &full[s], k * kK, int(tile.v0));
                        if (tile.width == kRows)
                            tma_load_2d(sx + C::kXBytes + kWBytes / 2, &tm_w, &full[s], k * kK, int(tile.v0) + 128);
                        for (int j = 0; j < wt; ++j)
                            bulk_load(sc + (1 + j) * mx::kTileBytes, ws + (int64_t(j) * a.k_tiles + k) * mx::kTileBytes,
                                      mx::kTileBytes, &full[s]);
                        tma_load_2d(sx, &tm_x, &full[s], k * kK, int(tile.n0));
                        bulk_load(sc, xs + int64_t(k) * mx::kTileBytes, mx::kTileBytes, &full[s]);
                    }
                }
                __syncwarp();
                issued |= 1u << s;
                issued_phase = (issued_phase & ~(1u << s)) | (phase << s);
                if (++s == uint32_t(S)) s = 0, phase ^= 1u;
            }
        }
        if (!ok)  // copies in flight land before shared memory is released
            for (int i = 0; i < S; ++i)
                if ((issued >> i) & 1u) mbar_wait(&full[i], (issued_phase >> i) & 1u, &no_abort, kDrainTimeoutNs);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        // What the instructions take is computed by the whole warp, outside the one lane's
        // branch, so that it sits in uniform registers: moved there one by one, the operands
        // of the seven instructions of a stage cost 660 clocks, now 410.
        uint32_t s = 0, phase = 0, acc = 0, acc_phase = 0, shared_phase = 0;
        const uint32_t sfa = tmem + kScaleCol, sfb = sfa + 4;
        const uint32_t x_lo = (smem_u32(smem) >> 4) | kTileLow, sc_lo = (smem_u32(scales) >> 4) | kScaleLow;
        const uint32_t empty_at = smem_u32(empty);
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int width = tile_at(a, t).width;
            if (!warp_wait(&t_empty[acc], acc_phase ^ 1u, abort_flag, a.timeout_ns)) break;
            if (!warp_wait(shared_empty, shared_phase ^ 1u, abort_flag, a.timeout_ns)) break;
            shared_phase ^= 1u;
            tc_fence_after();
            const uint32_t d = tmem + acc * kAccStep;
            const uint32_t idesc = width == kRows ? idesc_mx(kRows, 0) : idesc_mx(128, 0);
            for (int k = 0; k < a.k_tiles; ++k) {
                ok = warp_wait(&full[s], phase, abort_flag, a.timeout_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sc = sc_lo + s * (C::kScales >> 4);
                const uint32_t ax = x_lo + s * (C::kStage >> 4), bw = ax + (C::kXBytes >> 4);
                const uint32_t done = empty_at + s * 8;
                if (elect_one()) {
                    // copies to tensor memory and MMAs of one thread run in the order of issue
                    copy_scales(sfa, sc);
                    copy_scales(sfb, sc + (mx::kTileBytes >> 4));
                    if (width == kRows) copy_scales(sfb + 4, sc + 2 * (mx::kTileBytes >> 4));
                    umma_mx(d, ax, bw, idesc, sfa, sfb, k);
#pragma unroll
                    for (int kk = 1; kk < 4; ++kk)
                        umma_mx(d, ax + kk * 2, bw + kk * 2, idesc + kk * kScaleIdStep, sfa, sfb, 1u);
                    umma_commit(done);
                }
                __syncwarp();
                if (++s == uint32_t(S)) s = 0, phase ^= 1u;
            }
            if (!ok) break;
            if (elect_one()) umma_commit(smem_u32(&t_full[acc]));
            __syncwarp();
            acc ^= 1u;
            acc_phase ^= acc ^ 1u;
        }
        if (elect_one()) umma_commit(smem_u32(drain));  // every MMA completes before tensor memory is released
        __syncwarp();
        mbar_wait(drain, 0, &no_abort, kDrainTimeoutNs);
    } else if (warp >= kFirstEpilogue) {
        // ---------------- epilogue: one token per lane, 128 logits per warp ----------------
        const int ew = warp - kFirstEpilogue, q = warp & 3, half = ew >> 2;
        float* mine = reinterpret_cast<float*>(turn + ew * kTurnBytes);
        uint32_t acc = 0, acc_phase = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            if (!warp_wait(&t_full[acc], acc_phase, abort_flag, a.timeout_ns)) break;
            tc_fence_after();
            const Tile tile = tile_at(a, t);
            const int64_t n0 = tile.n0 + q * 32, v0 = tile.v0 + half * 128;
            store_tile<Out>(a, n0, v0, tile.v0 + tile.width, tmem + acc * kAccStep, acc, q, half, mine,
                            [&] { mbar_arrive(shared_empty); });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t_empty[acc]);
            acc ^= 1u;
            acc_phase ^= acc ^ 1u;
        }
    }

    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) report(a.dev_status, VCE_DEVSTATUS_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// CTA pairs
// ---------------------------------------------------------------------------

// The same for more than 128 tokens: two CTAs of a cluster take 256 tokens, 128 each, by 256
// classifier rows, of which each holds half in its shared memory; the even one issues the
// MMAs (cta_group::2) for both.  What a CTA writes and reads of shared memory per stage of
// 128 columns falls from 96 KB (768 clocks at 128 bytes per clock, which is what bound the
// kernel above) to 64 KB, below the tensor core's own time.
struct PairCfg {
    static constexpr uint32_t kXBytes = 128 * kK, kWHalf = 128 * kK;  // as the tensor core reads them
    static constexpr uint32_t kStage = kXBytes + kWHalf;
    static constexpr uint32_t kScales = 3 * mx::kTileBytes;  // the CTA's tokens', all 256 rows'
    static constexpr uint32_t kTx = 2 * (kXBytes + 128 * (kK / 2) + kScales);  // bytes a stage's copies count
    static constexpr int kStages = 6;
    static constexpr size_t kSmem = size_t(kStages) * (kStage + kScales) + kEpilogueWarps * kTurnBytes + 1024 + 512;
    static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint32_t low) {  // in both CTAs, from their own memory
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\ttcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(low), "n"(kScaleHigh)
        : "memory");
}

__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kTileHigh)
        : "memory");
}

template <typename Out>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mx_linear_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_xs,
                      const LinearArgs a) {
    using C = PairCfg;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* scales = smem + size_t(S) * C::kStage;
    uint8_t* turn = scales + size_t(S) * C::kScales;
    uint64_t* full = reinterpret_cast<uint64_t*>(turn + kEpilogueWarps * kTurnBytes);  // the even CTA's is used
    uint64_t* empty = full + S;
    uint64_t* t_full = empty + S;
    uint64_t* t_empty = t_full + 2;        // the even CTA's
    uint64_t* shared_empty = t_empty + 2;  // the even CTA's
    uint64_t* drain = shared_empty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int tiles = a.tiles_v * a.tiles_n, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], 2 * kEpilogueWarps);
        }
        mbar_init(shared_empty, 2 * 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // both CTAs' barriers exist before the first signal from one to the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int no_abort = 0;

    if (warp == 0) {
        // ---------------- copies, each CTA its own; all count on the even CTA's barriers ----------------
        if (lane == 0) {
            tma_prefetch_desc(&tm_w);
            tma_prefetch_desc(&tm_x);
            tma_prefetch_desc(&tm_ws);
            tma_prefetch_desc(&tm_xs);
        }
        uint32_t s = 0, phase = 0, issued = 0, issued_phase = 0;
        const uint32_t full_at = mapa_shared(smem_u32(full), 0);
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            const int tv = t / a.tiles_n, tn = t - tv * a.tiles_n;
            const int64_t v0 = int64_t(tv) * kRows, n0 = (int64_t(tn) * 2 + rank) * kTokens;
            // rows past the last come as zeros, for scales too; all of them count as bytes
            const int w_row = int(v0) + int(rank) * 128;
            const int ws = int(v0 / 128 * a.k_tiles * 2), xs = int(n0 / 128 * a.k_tiles * 2);
            for (int k = 0; k < a.k_tiles; ++k) {
                ok = warp_wait(&empty[s], phase ^ 1u, abort_flag, a.timeout_ns);
                if (!ok) break;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], C::kTx);
                    const uint32_t sx = smem_u32(smem + size_t(s) * C::kStage);
                    const uint32_t sc = smem_u32(scales + size_t(s) * C::kScales);
                    const uint32_t bar = full_at + s * 8;
                    if (VCE_BOUNDS(v0 < a.v && tn * 2 * int64_t(kTokens) < a.n && ws >= 0 && xs >= 0, a.dev_status)) {
                        tma_load_2d_pair(sx + C::kXBytes, &tm_w, bar, k * kK, w_row);
                        tma_load_2d_pair(sc + mx::kTileBytes, &tm_ws, bar, 0, ws + k * 2);
                        tma_load_2d_pair(sc + 2 * mx::kTileBytes, &tm_ws, bar, 0, ws + (a.k_tiles + k) * 2);
                        tma_load_2d_pair(sx, &tm_x, bar, k * kK, int(n0));
                        tma_load_2d_pair(sc, &tm_xs, bar, 0, xs + k * 2);
                    }
                }
                __syncwarp();
                issued |= 1u << s;
                issued_phase = (issued_phase & ~(1u << s)) | (phase << s);
                if (++s == uint32_t(S)) s = 0, phase ^= 1u;
            }
        }
        if (!ok && rank == 0)  // copies in flight land before shared memory is released
            for (int i = 0; i < S; ++i)
                if ((issued >> i) & 1u) mbar_wait(&full[i], (issued_phase >> i) & 1u, &no_abort, kDrainTimeoutNs);
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer ----------------
        uint32_t s = 0, phase = 0, acc = 0, acc_phase = 0, shared_phase = 0;
        const uint32_t sfa = tmem + kScaleCol, sfb = sfa + 4;
        const uint32_t x_lo = (smem_u32(smem) >> 4) | kTileLow, sc_lo = (smem_u32(scales) >> 4) | kScaleLow;
        constexpr uint32_t idesc = idesc_mx(kRows, 0) + (uint32_t(kTokens >> 4) << 24);  // M = 256
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            if (!warp_wait<true>(&t_empty[acc], acc_phase ^ 1u, abort_flag, a.timeout_ns)) break;
            if (!warp_wait<true>(shared_empty, shared_phase ^ 1u, abort_flag, a.timeout_ns)) break;
            shared_phase ^= 1u;
            tc_fence_after();
            const uint32_t d = tmem + acc * kAccStep;
            for (int k = 0; k < a.k_tiles; ++k) {
                ok = warp_wait(&full[s], phase, abort_flag, a.timeout_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sc = sc_lo + s * (C::kScales >> 4);
                const uint32_t ax = x_lo + s * (C::kStage >> 4), bw = ax + (C::kXBytes >> 4);
                if (elect_one()) {
                    copy_scales_pair(sfa, sc);
                    copy_scales_pair(sfb, sc + (mx::kTileBytes >> 4));
                    copy_scales_pair(sfb + 4, sc + 2 * (mx::kTileBytes >> 4));
                    umma_mx_pair(d, ax, bw, idesc, sfa, sfb, k);
#pragma unroll
                    for (int kk = 1; kk < 4; ++kk)
                        umma_mx_pair(d, ax + kk * 2, bw + kk * 2, idesc + kk * kScaleIdStep, sfa, sfb, 1u);
                    umma_commit_pair(&empty[s], 0x3);
                }
                __syncwarp();
                if (++s == uint32_t(S)) s = 0, phase ^= 1u;
            }
            if (!ok) break;
            if (elect_one()) umma_commit_pair(&t_full[acc], 0x3);
            __syncwarp();
            acc ^= 1u;
            acc_phase ^= acc ^ 1u;
        }
        if (elect_one()) umma_commit_pair(drain, 0x1);  // every MMA completes before tensor memory is released
        __syncwarp();
        mbar_wait(drain, 0, &no_abort, kDrainTimeoutNs);
    } else if (warp >= kFirstEpilogue) {
        const int ew = warp - kFirstEpilogue, q = warp & 3, half = ew >> 2;
        float* mine = reinterpret_cast<float*>(turn + ew * kTurnBytes);
        const uint32_t t_empty_at = mapa_shared(smem_u32(t_empty), 0);
        const uint32_t shared_at = mapa_shared(smem_u32(shared_empty), 0);
        uint32_t acc = 0, acc_phase = 0;
        for (int t = pair; t < tiles; t += pairs) {
            if (!warp_wait(&t_full[acc], acc_phase, abort_flag, a.timeout_ns)) break;
            tc_fence_after();
            const int tv = t / a.tiles_n, tn = t - tv * a.tiles_n;
            const int64_t v0 = int64_t(tv) * kRows, n0 = (int64_t(tn) * 2 + rank) * kTokens + q * 32;
            store_tile<Out>(a, n0, v0 + half * 128, v0 + kRows, tmem + acc * kAccStep, acc, q, half, mine,
                            [&] { mbar_arrive_cluster(shared_at); });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(t_empty_at + acc * 8);
            acc ^= 1u;
            acc_phase ^= acc ^ 1u;
        }
    }

    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) report(a.dev_status, VCE_DEVSTATUS_TIMEOUT);
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // no more MMAs, copies or signals from the other CTA
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Codes [rows][cols], box of 128 columns x ``box_rows``, 128-byte swizzle, zeros out of
// range.  E2M1 codes are spread to one byte per value's place (see above); that type
// wants columns and x coordinates in multiples of 128 and the base at 32 bytes.
bool code_map(CUtensorMap* map, const void* base, bool packed, uint64_t cols, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {packed ? cols / 2 : cols};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t es[2] = {1, 1};
    return fn(map, packed ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
              const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 256 bytes, two to a tile.
bool scale_map(CUtensorMap* map, const void* base, uint64_t tiles) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {256, tiles * 2};
    cuuint64_t strides[1] = {256};
    cuuint32_t box[2] = {256, 2};
    cuuint32_t es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Out>
vce_status launch_pair(const void* xc, const void* wc, LinearArgs a, cudaStream_t s, const DeviceInfo& dev) {
    static std::mutex mu;
    static bool ready[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev.ordinal]) {
            if (cudaFuncSetAttribute(mx_linear_pair_kernel<Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(PairCfg::kSmem)) != cudaSuccess)
                return VCE_ERR_CUDA;
            ready[dev.ordinal] = true;
        }
    }
    CUtensorMap tm_w, tm_x, tm_ws, tm_xs;
    const uint64_t cols = uint64_t(a.k_tiles) * kK;
    if (!code_map(&tm_w, wc, true, cols, uint64_t(a.v), 128) || !code_map(&tm_x, xc, false, cols, uint64_t(a.n), 128) ||
        !scale_map(&tm_ws, a.w_scales, uint64_t(a.w_scale_rows) * a.k_tiles) ||
        !scale_map(&tm_xs, a.x_scales, uint64_t((a.n + 127) / 128) * a.k_tiles))
        return VCE_ERR_CUDA;
    const int64_t tiles = int64_t(a.tiles_v) * a.tiles_n;
    count_launch();
    mx_linear_pair_kernel<Out><<<2 * unsigned(tiles < dev.num_sms / 2 ? tiles : dev.num_sms / 2), kThreads,
                                 PairCfg::kSmem, s>>>(tm_w, tm_x, tm_ws, tm_xs, a);
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

template <int XR, typename Out>
vce_status launch(const void* xc, const void* wc, LinearArgs a, cudaStream_t s, const DeviceInfo& dev) {
    static std::mutex mu;
    static bool ready[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev.ordinal]) {
            if (cudaFuncSetAttribute(mx_linear_kernel<XR, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(Cfg<XR>::kSmem)) != cudaSuccess)
                return VCE_ERR_CUDA;
            ready[dev.ordinal] = true;
        }
    }
    CUtensorMap tm_w, tm_x;
    const uint64_t cols = uint64_t(a.k_tiles) * kK;
    if (!code_map(&tm_w, wc, true, cols, uint64_t(a.v), 128) || !code_map(&tm_x, xc, false, cols, uint64_t(a.n), XR))
        return VCE_ERR_CUDA;
    const int64_t tiles = int64_t(a.tiles_v) * a.tiles_n;
    if (tiles > 0x7fffffff) return VCE_ERR_INVALID_ARG;
    count_launch();
    mx_linear_kernel<XR, Out><<<unsigned(tiles < dev.num_sms ? tiles : dev.num_sms), kThreads, Cfg<XR>::kSmem, s>>>(
        tm_w, tm_x, a);
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

template <typename Out>
vce_status dispatch(const void* xc, const void* wc, LinearArgs a, cudaStream_t s, const DeviceInfo& dev) {
    const int64_t at = int64_t(reinterpret_cast<uintptr_t>(a.out)) | a.out_stride * int64_t(sizeof(Out));
    a.wide = at % 32 == 0 ? 2 : at % 16 == 0 ? 1 : 0;
    const mx::LinearPlan p = mx::plan_linear(a.n, a.v, a.k_tiles, dev.num_sms);
    a.tiles_n = int(p.tiles_n), a.tiles_v = int(p.tiles_v), a.whole_v = int(p.whole_v);
    if (p.pairs) return launch_pair<Out>(xc, wc, a, s, dev);
    if (a.n <= 16) return launch<16, Out>(xc, wc, a, s, dev);
    if (a.n <= 64) return launch<64, Out>(xc, wc, a, s, dev);
    return launch<128, Out>(xc, wc, a, s, dev);
}

}  // namespace

vce_status launch_mx_linear(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                            int64_t n, int64_t v, int64_t h, void* out, int out_dtype, int64_t out_stride,
                            int* dev_status, cudaStream_t s, const DeviceInfo& dev) {
    if (n == 0) return VCE_OK;
    LinearArgs a{};
    a.n = n; a.v = v; a.k_tiles = int(mx::padded(h) / kK);
    a.w_scales = static_cast<const uint8_t*>(w_scales);
    a.x_scales = static_cast<const uint8_t*>(x_scales);
    a.w_scale_rows = mx::padded(v) / mx::kRowTile;
    a.out = out; a.out_stride = out_stride; a.dev_status = dev_status; a.timeout_ns = kPipeTimeoutNs;
    return out_dtype == VCE_BF16 ? dispatch<__nv_bfloat16>(x_codes, w_codes, a, s, dev)
                                 : dispatch<float>(x_codes, w_codes, a, s, dev);
}

}  // namespace vce
