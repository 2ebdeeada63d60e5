// Product of microscaled matrices: logits[n, v] = sum_k x[n, k] w[v, k], x in E4M3 and
// the classifier w in E2M1, each with one power-of-two scale per 32 values of k.
//
// tcgen05.mma.kind::mxf8f6f4 with block scales multiplies such operands as they are:
// products of codes are exact, the two scales of a block of 32 are applied inside the
// tensor core and sums are FP32.  Tokens are the M operand (128 of them, one per
// tensor-memory lane) and the classifier's rows the N operand, for few tokens too: an
// instruction with N = 16 tokens over 128 classifier rows costs nearly as much as one
// with N = 128, and the classifier is what has to be fed through (8 tokens x 4096 x
// 128256: 120 us that way round).
//
// 4-bit values travel packed (two per byte) from HBM to shared memory.  The tensor
// core wants them there as 16-byte pieces of 16 values, 8 bytes of codes and 8 of
// padding; converter warps spread the codes from the packed ring into the operand ring.
//
// Roles: warp 0 copies packed w and its scales (TMA), warp 1 issues the MMAs, warp 2
// copies x and its scales, then epilogue warps and converters.  Three rings: ``packed``
// (256 columns of w per stage, the bytes that come from HBM, kept deep), ``w`` (128
// columns, converted) and ``x`` (128 columns).  Every wait is bounded, as in lce_tc.cu.

#include "vce_internal.cuh"
#include "mx_format.cuh"
#include "sm100_ptx.cuh"

#include <cudaTypedefs.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kTokens = 128;                    // tokens per tile
constexpr int kK = 128;                         // columns per operand stage: one 128-byte swizzle row
constexpr int kPackedK = 256;                   // columns per packed stage: 128-byte rows, too
constexpr uint32_t kXBytes = kTokens * kK;
constexpr int kFirstEpilogue = 4;               // warp; a multiple of 4, as lane quadrants go by warp % 4
constexpr int kStageCols = 16;                  // columns an epilogue warp turns at a time
constexpr uint32_t kTurnBytes = 32 * (kStageCols + 1) * 4;  // and its scratch

// BN: classifier rows per tile
template <int BN>
struct Cfg {
    static constexpr int kWTiles = BN / 128;                 // scale tiles of w
    static constexpr uint32_t kWBytes = BN * kK;             // converted
    static constexpr uint32_t kPackedBytes = BN * kPackedK / 2;
    static constexpr uint32_t kPackedScales = 2 * kWTiles * mx::kTileBytes;
    static constexpr int kW = BN == 128 ? 3 : 2;             // stages
    static constexpr int kX = 3;
    static constexpr int kPacked = BN == 128 ? 5 : 2;
    static constexpr int kAccs = BN == 128 ? 2 : 1;
    static constexpr int kEpilogueWarps = BN / 32;           // four per 128 columns
    static constexpr int kConverterWarps = BN / 32;          // 32 rows each
    static constexpr int kFirstConverter = kFirstEpilogue + kEpilogueWarps;
    static constexpr int kThreads = (kFirstConverter + kConverterWarps) * 32;
    static constexpr uint32_t kScaleCol = kAccs * BN;        // tensor-memory column of x's scales, w's behind
    static constexpr uint32_t kTmemCols = 512;
    static constexpr size_t kSmem = size_t(kW) * (kWBytes + kWTiles * mx::kTileBytes) +
                                    size_t(kX) * (kXBytes + mx::kTileBytes) +
                                    size_t(kPacked) * (kPackedBytes + kPackedScales) + kEpilogueWarps * kTurnBytes +
                                    1024 + 512;
    static_assert(kScaleCol + 4 + 4 * kWTiles <= kTmemCols && kSmem <= 232448, "tensor and shared memory");
};

struct LinearArgs {
    int64_t n, v;
    int k_tiles;           // 128-column tiles
    int tiles_v, tiles_n;
    int x_rows;            // tokens per copy of x: 16, 32, 64 or 128
    int64_t w_scale_rows;  // 128-row tiles of w's scales
    const uint8_t *w_scales, *x_scales;
    void* out;
    int64_t out_stride;
    int wide;              // every 32 columns of a row start 16-byte aligned
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
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, timeout_ns));
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 32 consecutive logits of one token, 16-byte aligned
__device__ __forceinline__ void store_row32(float* p, const uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
}
__device__ __forceinline__ void store_row32(__nv_bfloat16* p, const uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * k]),
                                                           __uint_as_float(r[8 * i + 2 * k + 1]));
            u[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        reinterpret_cast<uint4*>(p)[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

template <int BN, typename Out>
__global__ void __launch_bounds__(Cfg<BN>::kThreads, 1)
mx_linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                 const LinearArgs a) {
    using C = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* w_ring = smem;                                           // operand tiles and packed ones: 1024-aligned
    uint8_t* packed = w_ring + size_t(C::kW) * C::kWBytes;
    uint8_t* x_ring = packed + size_t(C::kPacked) * C::kPackedBytes;
    uint8_t* packed_scales = x_ring + size_t(C::kX) * kXBytes;
    uint8_t* w_scales = packed_scales + size_t(C::kPacked) * C::kPackedScales;
    uint8_t* x_scales = w_scales + size_t(C::kW) * C::kWTiles * mx::kTileBytes;
    uint8_t* turn = x_scales + size_t(C::kX) * mx::kTileBytes;
    uint64_t* p_full = reinterpret_cast<uint64_t*>(turn + C::kEpilogueWarps * kTurnBytes);
    uint64_t* p_empty = p_full + C::kPacked;  // read by the converter warps
    uint64_t* w_full = p_empty + C::kPacked;  // converted by them
    uint64_t* w_empty = w_full + C::kW;       // MMAs done with the stage
    uint64_t* x_full = w_empty + C::kW;
    uint64_t* x_empty = x_full + C::kX;
    uint64_t* t_full = x_empty + C::kX;
    uint64_t* t_empty = t_full + 2;
    uint64_t* drain = t_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = a.tiles_v * a.tiles_n;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kPacked; ++i) {
            mbar_init(&p_full[i], 1);
            mbar_init(&p_empty[i], C::kConverterWarps);
        }
        for (int i = 0; i < C::kW; ++i) {
            mbar_init(&w_full[i], C::kConverterWarps);
            mbar_init(&w_empty[i], 1);
        }
        for (int i = 0; i < C::kX; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], C::kEpilogueWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // Rows of x that no copy writes (fewer tokens than a tile): zeros for the whole launch
    if (a.x_rows < kTokens) {
        for (int s = 0; s < C::kX; ++s)
            for (int i = a.x_rows * 8 + threadIdx.x; i < int(kXBytes / 16); i += C::kThreads)
                reinterpret_cast<uint4*>(x_ring + size_t(s) * kXBytes)[i] = make_uint4(0, 0, 0, 0);
        fence_async_shared();
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int no_abort = 0;

    if (warp == 0) {
        {
            // ---------------- packed w and its scales ----------------
            if (lane == 0) tma_prefetch_desc(&tm_w);
            uint32_t s = 0, phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int tv = t / a.tiles_n;
                const int64_t tile0 = int64_t(tv) * C::kWTiles;
                const int wt = int(a.w_scale_rows - tile0 < C::kWTiles ? a.w_scale_rows - tile0 : C::kWTiles);
                for (int k = 0; k < a.k_tiles; k += 2) {
                    if (!warp_wait(&p_empty[s], phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sb = (k + 1 < a.k_tiles ? 2 : 1) * mx::kTileBytes;
                    // past the last column and row the copies read zeros
                    if (lane == 0) mbar_arrive_expect_tx(&p_full[s], C::kPackedBytes + wt * sb);
                    if (lane == 0 && VCE_BOUNDS(k * (kK / 2) % 16 == 0 && tv < a.tiles_v && wt >= 1, a.dev_status)) {
#pragma unroll
                        for (int j = 0; j < C::kWTiles; ++j)
                            tma_load_2d(smem_u32(packed + size_t(s) * C::kPackedBytes + j * 128 * (kPackedK / 2)), &tm_w,
                                        &p_full[s], k * (kK / 2), tv * BN + j * 128);
                        for (int j = 0; j < wt; ++j)
                            bulk_load(smem_u32(packed_scales + size_t(s) * C::kPackedScales + j * 2 * mx::kTileBytes),
                                      a.w_scales + ((tile0 + j) * a.k_tiles + k) * mx::kTileBytes, sb, &p_full[s]);
                    }
                    issued |= 1u << s;
                    issued_phase = (issued_phase & ~(1u << s)) | (phase << s);
                    if (++s == uint32_t(C::kPacked)) s = 0, phase ^= 1u;
                }
            }
            if (!ok)  // copies in flight land before shared memory is released
                for (int i = 0; i < C::kPacked; ++i)
                    if ((issued >> i) & 1u) mbar_wait(&p_full[i], (issued_phase >> i) & 1u, &no_abort, kDrainTimeoutNs);
        }
    } else if (warp == 2) {
        {
            // ---------------- x and its scales ----------------
            if (lane == 0) tma_prefetch_desc(&tm_x);
            uint32_t s = 0, phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int tn = t % a.tiles_n;
                for (int k = 0; k < a.k_tiles; ++k) {
                    if (!warp_wait(&x_empty[s], phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&x_full[s], a.x_rows * kK + mx::kTileBytes);
                    if (lane == 0 && VCE_BOUNDS(tn < a.tiles_n && a.x_rows <= kTokens, a.dev_status)) {
                        tma_load_2d(smem_u32(x_ring + size_t(s) * kXBytes), &tm_x, &x_full[s], k * kK, tn * kTokens);
                        bulk_load(smem_u32(x_scales + size_t(s) * mx::kTileBytes),
                                  a.x_scales + (int64_t(tn) * a.k_tiles + k) * mx::kTileBytes, mx::kTileBytes,
                                  &x_full[s]);
                    }
                    issued |= 1u << s;
                    issued_phase = (issued_phase & ~(1u << s)) | (phase << s);
                    if (++s == uint32_t(C::kX)) s = 0, phase ^= 1u;
                }
            }
            if (!ok)
                for (int i = 0; i < C::kX; ++i)
                    if ((issued >> i) & 1u) mbar_wait(&x_full[i], (issued_phase >> i) & 1u, &no_abort, kDrainTimeoutNs);
        }
    } else if (warp == 1) {
        {
            // ---------------- MMA issuer ----------------
            uint32_t sw = 0, w_phase = 0, sx = 0, x_phase = 0, acc = 0, acc_phase = 0;
            const uint32_t sfa = tmem + C::kScaleCol, sfb = sfa + 4;
            const uint32_t x_lo = (smem_u32(x_ring) >> 4) | kTileLow, w_lo = (smem_u32(w_ring) >> 4) | kTileLow;
            const uint32_t x_sc = (smem_u32(x_scales) >> 4) | kScaleLow, w_sc = (smem_u32(w_scales) >> 4) | kScaleLow;
            const uint32_t w_bar = smem_u32(w_empty), x_bar = smem_u32(x_empty);
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                if (!warp_wait(&t_empty[acc], acc_phase ^ 1u, abort_flag, a.timeout_ns)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                for (int k = 0; k < a.k_tiles; ++k) {
                    if (
                        !warp_wait(&x_full[sx], x_phase, abort_flag, a.timeout_ns) ||
                        !warp_wait(&w_full[sw], w_phase, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // copies to tensor memory and MMAs of one thread run in the order of issue
                    const uint32_t xs = x_sc + sx * (mx::kTileBytes >> 4);
                    const uint32_t ws = w_sc + sw * (C::kWTiles * mx::kTileBytes >> 4);
                    const uint32_t ax = x_lo + sx * (kXBytes >> 4), bw = w_lo + sw * (C::kWBytes >> 4);
                    const uint32_t we = w_bar + sw * 8, xe = x_bar + sx * 8;
                    if (elect_one()) {
                        copy_scales(sfa, xs);
#pragma unroll
                        for (int j = 0; j < C::kWTiles; ++j) copy_scales(sfb + 4 * j, ws + j * (mx::kTileBytes >> 4));
                        umma_mx(d, ax, bw, idesc_mx(BN, 0), sfa, sfb, k);
#pragma unroll
                        for (int kk = 1; kk < 4; ++kk)
                            umma_mx(d, ax + kk * 2, bw + kk * 2, idesc_mx(BN, kk), sfa, sfb, 1u);
                        umma_commit(we);
                        umma_commit(xe);
                    }
                    __syncwarp();
                    if (++sw == uint32_t(C::kW)) sw = 0, w_phase ^= 1u;
                    if (++sx == uint32_t(C::kX)) sx = 0, x_phase ^= 1u;
                }
                if (!ok) break;
                if (elect_one()) umma_commit(smem_u32(&t_full[acc]));
                __syncwarp();
                if (++acc == uint32_t(C::kAccs)) acc = 0, acc_phase ^= 1u;
            }
            if (elect_one()) umma_commit(smem_u32(drain));
            __syncwarp();  // every MMA completes before tensor memory is released
            mbar_wait(drain, 0, &no_abort, kDrainTimeoutNs);
        }
    } else if (warp >= C::kFirstConverter) {
        // ---------------- converters: 32 classifier rows per warp ----------------
        // A lane takes 16 packed bytes (32 values) of a row and stores them as two
        // 16-byte pieces with 8 bytes of codes each.  Both rings use the 128-byte swizzle
        // (piece p of row r at p ^ (r & 7)).  Lanes 0-3 read four neighbouring pieces of
        // one row and lanes 4-7 those of the row four further, which the swizzle puts in
        // the other half of the banks.
        const int cw = warp - C::kFirstConverter;
        const int sub = lane & 3, row0 = cw * 32 + ((lane >> 2) & 1) * 4 + (lane >> 3), x = row0 & 7;
        // byte offsets in a tile of this lane's piece of its first row (the others are 1024
        // further each): packed, for either half of the stage, and the two converted pieces
        const uint32_t from[2] = {uint32_t(row0 * 128 + ((sub ^ x) << 4)), uint32_t(row0 * 128 + (((4 + sub) ^ x) << 4))};
        const uint32_t to0 = row0 * 128 + (((2 * sub) ^ x) << 4), to1 = row0 * 128 + (((2 * sub + 1) ^ x) << 4);
        uint32_t ps = 0, p_phase = 0, s = 0, phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            for (int k = 0; k < a.k_tiles && ok; k += 2) {
                ok = warp_wait(&p_full[ps], p_phase, abort_flag, a.timeout_ns);
                if (!ok) break;
                const uint8_t* src = packed + size_t(ps) * C::kPackedBytes;
                const int halves = k + 1 < a.k_tiles ? 2 : 1;
                for (int h = 0; h < halves; ++h) {
                    uint4 q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const uint4*>(src + (h ? from[1] : from[0]) + i * 1024);
                    // a quarter of a scale tile: tile cw / 4, its words 32 (cw % 4) ...
                    const uint32_t sc = reinterpret_cast<const uint32_t*>(
                        packed_scales + size_t(ps) * C::kPackedScales +
                        ((cw >> 2) * 2 + h) * mx::kTileBytes)[(cw & 3) * 32 + lane];
                    ok = warp_wait(&w_empty[s], phase ^ 1u, abort_flag, a.timeout_ns);
                    if (!ok) break;
                    uint8_t* dst = w_ring + size_t(s) * C::kWBytes;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *reinterpret_cast<uint2*>(dst + to0 + i * 1024) = make_uint2(q[i].x, q[i].y);
                        *reinterpret_cast<uint2*>(dst + to1 + i * 1024) = make_uint2(q[i].z, q[i].w);
                    }
                    reinterpret_cast<uint32_t*>(w_scales + size_t(s) * C::kWTiles * mx::kTileBytes)[cw * 32 + lane] = sc;
                    fence_async_shared();  // the tensor core reads these through the async proxy
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&w_full[s]);
                        // only now: loads whose values have been stored are certainly over, and the
                        // next copy into the packed stage cannot overtake them
                        if (h + 1 == halves) mbar_arrive(&p_empty[ps]);
                    }
                    if (++s == uint32_t(C::kW)) s = 0, phase ^= 1u;
                }
                if (++ps == uint32_t(C::kPacked)) ps = 0, p_phase ^= 1u;
            }
        }
    } else if (warp >= kFirstEpilogue) {
        // ---------------- epilogue: one token per lane, 128 logits per warp ----------------
        const int ew = warp - kFirstEpilogue, q = warp & 3, col0 = (ew >> 2) * 128;
        float* mine = reinterpret_cast<float*>(turn + ew * kTurnBytes);
        uint32_t acc = 0, acc_phase = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            if (!warp_wait(&t_full[acc], acc_phase, abort_flag, a.timeout_ns)) break;
            tc_fence_after();
            const int64_t n0 = int64_t(t % a.tiles_n) * kTokens + q * 32;
            const int64_t v0 = int64_t(t / a.tiles_n) * BN + col0;
            const int live = int(a.n - n0 < 32 ? a.n - n0 : 32);  // tokens of this warp
            const int cols = int(a.v - v0 < 128 ? a.v - v0 : 128);
            const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + acc * BN + col0;
            Out* out = static_cast<Out*>(a.out) + n0 * a.out_stride + v0;
            if (live > 0 && cols > 0 && VCE_BOUNDS(n0 >= 0 && v0 >= 0, a.dev_status)) {
                if (a.wide) {
                    Out* row = out + int64_t(lane) * a.out_stride;
#pragma unroll 1
                    for (int c = 0; c < cols; c += 32) {
                        uint32_t r[32];
                        tmem_ld32(taddr + c, r);
                        tmem_ld_wait();
                        if (lane < live) {
                            if (cols - c >= 32) {
                                store_row32(row + c, r);
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (j < cols - c) store_logit(row + c + j, __uint_as_float(r[j]));
                            }
                        }
                    }
                } else {
                    // rows at any offset: turned through shared memory, so that half a warp
                    // stores 16 neighbouring logits of one token
                    const int hl = lane & 15, hr = lane >> 4;
#pragma unroll 1
                    for (int c = 0; c < cols; c += 32) {
                        uint32_t r[32];
                        tmem_ld32(taddr + c, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < kStageCols; ++j)
                                mine[lane * (kStageCols + 1) + j] = __uint_as_float(r[part * kStageCols + j]);
                            __syncwarp();
                            const int cc = c + part * kStageCols + hl;
                            if (cc < cols) {
                                Out* p = out + int64_t(hr) * a.out_stride + cc;
                                for (int i = hr; i < live; i += 2, p += 2 * a.out_stride)
                                    store_logit(p, mine[i * (kStageCols + 1) + hl]);
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t_empty[acc]);
            if (++acc == uint32_t(C::kAccs)) acc = 0, acc_phase ^= 1u;
        }
    }

    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) report(a.dev_status, VCE_DEVSTATUS_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
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

// Bytes [rows][row_bytes], box of 128 bytes x ``box_rows``, 128-byte swizzle, zeros out of range.
bool byte_map(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {row_bytes, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename Out>
vce_status launch(const void* xc, const void* wc, LinearArgs a, cudaStream_t s, const DeviceInfo& dev) {
    static std::mutex mu;
    static bool ready[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev.ordinal]) {
            if (cudaFuncSetAttribute(mx_linear_kernel<BN, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(Cfg<BN>::kSmem)) != cudaSuccess)
                return VCE_ERR_CUDA;
            ready[dev.ordinal] = true;
        }
    }
    CUtensorMap tm_w, tm_x;
    const uint64_t cols = uint64_t(a.k_tiles) * kK;
    if (!byte_map(&tm_w, wc, cols / 2, uint64_t(a.v), 128) || !byte_map(&tm_x, xc, cols, uint64_t(a.n), a.x_rows))
        return VCE_ERR_CUDA;
    a.tiles_v = int((a.v + BN - 1) / BN);
    const int64_t tiles = int64_t(a.tiles_v) * a.tiles_n;
    if (tiles > 0x7fffffff) return VCE_ERR_INVALID_ARG;
    count_launch();
    mx_linear_kernel<BN, Out>
        <<<unsigned(tiles < dev.num_sms ? tiles : dev.num_sms), Cfg<BN>::kThreads, Cfg<BN>::kSmem, s>>>(tm_w, tm_x, a);
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

template <typename Out>
vce_status dispatch(const void* xc, const void* wc, LinearArgs a, cudaStream_t s, const DeviceInfo& dev) {
    a.tiles_n = int((a.n + kTokens - 1) / kTokens);
    a.x_rows = a.n <= 16 ? 16 : a.n <= 32 ? 32 : a.n <= 64 ? 64 : kTokens;
    a.wide = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride * int64_t(sizeof(Out)) % 16 == 0;
#ifdef X_BN
    return launch<X_BN, Out>(xc, wc, a, s, dev);
#endif
    // 256 classifier rows per tile where that many tiles keep every SM busy
    const int64_t tiles = (a.v + 255) / 256 * a.tiles_n;
    if (tiles >= 8 * dev.num_sms) return launch<256, Out>(xc, wc, a, s, dev);
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
