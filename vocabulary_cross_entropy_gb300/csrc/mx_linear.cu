// Product of microscaled matrices: logits[n, v] = sum_k x[n, k] w[v, k], x in E4M3 and
// the classifier w in E2M1, each with one power-of-two scale per 32 values of k.
//
// tcgen05.mma.kind::mxf8f6f4 with block scales multiplies such operands as they are:
// products of codes are exact, the two scales of a block of 32 are applied inside the
// tensor core and sums are FP32.  The classifier is the M operand (128 vocabulary
// entries, one per tensor-memory lane) and the tokens the N operand, so that a few
// tokens cost a narrow N instead of a mostly empty M, and an epilogue warp stores 32
// neighbouring logits of one token at a time.
//
// 4-bit values travel packed (two per byte) from HBM to shared memory.  The tensor
// core wants them there as 16-byte pieces of 16 values, 8 bytes of codes and 8 of
// padding; converter warps spread the codes from the packed ring into the operand ring.
//
// Roles: warp 0 copies packed w and its scales (TMA), warp 1 issues the MMAs, warps
// 2-5 drain accumulators, warps 6-9 convert, warp 10 copies x and its scales.  Two
// rings: ``packed`` (256 columns of w per stage, the bytes that come from HBM, kept
// deep) and ``operand`` (128 columns of both, ready for the MMA).  Every wait is
// bounded, as in lce_tc.cu.

#include "vce_internal.cuh"
#include "mx_format.cuh"
#include "sm100_ptx.cuh"

#include <cudaTypedefs.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kRows = 128;                      // vocabulary entries per tile
constexpr int kK = 128;                         // columns per operand stage: one 128-byte swizzle row
constexpr int kPackedK = 256;                   // columns per packed stage
constexpr uint32_t kPackedBytes = kRows * kPackedK / 2;
constexpr uint32_t kPackedStage = kPackedBytes + 2 * mx::kTileBytes;
constexpr uint32_t kWBytes = kRows * kK;        // converted w of one operand stage
constexpr int kThreads = 352;

template <int BN>
struct Cfg {
    static constexpr uint32_t kXBytes = BN * kK;
    static constexpr int kXTiles = BN > 128 ? BN / 128 : 1;  // scale tiles of x
    static constexpr uint32_t kStage = kWBytes + kXBytes;    // a multiple of 1024
    static constexpr uint32_t kScales = mx::kTileBytes * (1 + kXTiles);
    static constexpr int kStages = BN <= 64 ? 5 : BN == 128 ? 4 : 3;
    static constexpr int kPacked = BN <= 32 ? 6 : BN <= 128 ? 5 : 4;
    static constexpr int kAccs = BN > 128 ? 1 : 2;
    static constexpr uint32_t kScaleCol = kAccs * BN;  // tensor-memory column of w's scales, x's behind
    static constexpr uint32_t kCols = kScaleCol + 4 + 4 * kXTiles;
    static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr size_t kSmem = size_t(kStages) * (kStage + kScales) + size_t(kPacked) * kPackedStage + 1024 + 512;
    static_assert(kCols <= 512 && kSmem <= 232448, "tensor and shared memory");
};

struct LinearArgs {
    int64_t n, v;
    int k_tiles;           // 128-column tiles
    int tiles_v, tiles_n;
    const uint8_t *w_scales, *x_scales;
    int64_t x_scale_rows;  // 128-row tiles of x's scales
    void* out;
    int64_t out_stride;
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

__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Descriptor of a scale tile in shared memory: 32 rows of 16 bytes without swizzle,
// 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t(128 >> 4) << 16 | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
}

// A 512-byte scale tile into four tensor-memory columns (rows 32 j .. 32 j + 31 in
// column j, a byte per 32 columns of k), repeated in all four lane quadrants.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: A E2M1 (5) at bit 7, B E4M3 (0) at bit 10,
// N >> 3 at bit 17, E8M0 scales (bit 23), M >> 4 at bit 24; the byte of the scale
// columns that holds this k step at bits 29 (A) and 4 (B).
__device__ constexpr uint32_t idesc_mx(int n, int k_step) {
    return (5u << 7) | (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(kRows >> 4) << 24) |
           (uint32_t(k_step) << 29) | (uint32_t(k_step) << 4);
}

__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int BN, typename Out>
__global__ void __launch_bounds__(kThreads, 1)
mx_linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                 const LinearArgs a) {
    using C = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* packed = smem + size_t(C::kStages) * C::kStage;                  // kPacked x 16 KiB (1024-aligned)
    uint8_t* packed_scales = packed + size_t(C::kPacked) * kPackedBytes;      // kPacked x 1 KiB
    uint8_t* scales = packed_scales + size_t(C::kPacked) * 2 * mx::kTileBytes;  // kStages x (w, x)
    uint64_t* p_full = reinterpret_cast<uint64_t*>(scales + size_t(C::kStages) * C::kScales);
    uint64_t* p_empty = p_full + C::kPacked;   // the four converter warps
    uint64_t* w_full = p_empty + C::kPacked;   // converted w and its scales: four converter warps
    uint64_t* x_full = w_full + C::kStages;    // x and its scales
    uint64_t* empty = x_full + C::kStages;     // MMAs done with the stage
    uint64_t* t_full = empty + C::kStages;
    uint64_t* t_empty = t_full + 2;
    uint64_t* drain = t_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = a.tiles_v * a.tiles_n;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kPacked; ++i) {
            mbar_init(&p_full[i], 1);
            mbar_init(&p_empty[i], 4);
        }
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&w_full[i], 4);
            mbar_init(&x_full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int no_abort = 0;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- packed w and its scales ----------------
            tma_prefetch_desc(&tm_w);
            uint32_t s = 0, phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int tv = t / a.tiles_n;
                for (int k = 0; k < a.k_tiles; k += 2) {
                    if (!mbar_wait(&p_empty[s], phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sb = (k + 1 < a.k_tiles ? 2 : 1) * mx::kTileBytes;
                    mbar_arrive_expect_tx(&p_full[s], kPackedBytes + sb);
                    // past the last column and row the copy reads zeros
                    if (VCE_BOUNDS(k * (kK / 2) % 16 == 0 && tv < a.tiles_v, a.dev_status)) {
                        tma_load_2d(smem_u32(packed + size_t(s) * kPackedBytes), &tm_w, &p_full[s], k * (kK / 2),
                                    tv * kRows);
                        bulk_load(smem_u32(packed_scales + size_t(s) * 2 * mx::kTileBytes),
                                  a.w_scales + (int64_t(tv) * a.k_tiles + k) * mx::kTileBytes, sb, &p_full[s]);
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
    } else if (warp == 10) {
        if (lane == 0) {
            // ---------------- x and its scales ----------------
            tma_prefetch_desc(&tm_x);
            uint32_t s = 0, phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int tn = t % a.tiles_n;
                const int64_t tile0 = int64_t(tn) * C::kXTiles;  // (BN below 128: one token tile)
                const int xt = int(a.x_scale_rows - tile0 < C::kXTiles ? a.x_scale_rows - tile0 : C::kXTiles);
                for (int k = 0; k < a.k_tiles; ++k) {
                    if (!mbar_wait(&empty[s], phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&x_full[s], C::kXBytes + xt * mx::kTileBytes);
                    if (VCE_BOUNDS(xt >= 1 && tn < a.tiles_n, a.dev_status)) {
                        tma_load_2d(smem_u32(smem + size_t(s) * C::kStage + kWBytes), &tm_x, &x_full[s], k * kK, tn * BN);
                        for (int j = 0; j < xt; ++j)
                            bulk_load(smem_u32(scales + size_t(s) * C::kScales + (1 + j) * mx::kTileBytes),
                                      a.x_scales + ((tile0 + j) * a.k_tiles + k) * mx::kTileBytes, mx::kTileBytes,
                                      &x_full[s]);
                    }
                    issued |= 1u << s;
                    issued_phase = (issued_phase & ~(1u << s)) | (phase << s);
                    if (++s == uint32_t(C::kStages)) s = 0, phase ^= 1u;
                }
            }
            if (!ok)
                for (int i = 0; i < C::kStages; ++i)
                    if ((issued >> i) & 1u) mbar_wait(&x_full[i], (issued_phase >> i) & 1u, &no_abort, kDrainTimeoutNs);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            uint32_t s = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                if (!mbar_wait(&t_empty[acc], acc_phase ^ 1u, abort_flag, a.timeout_ns)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * BN, sfa = tmem + C::kScaleCol, sfb = sfa + 4;
                for (int k = 0; k < a.k_tiles; ++k) {
                    if (!mbar_wait(&x_full[s], phase, abort_flag, a.timeout_ns) ||
                        !mbar_wait(&w_full[s], phase, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // copies to tensor memory and MMAs of one thread run in the order of issue
                    const uint32_t sc = smem_u32(scales + size_t(s) * C::kScales);
                    copy_scales(sfa, scale_desc(sc));
#pragma unroll
                    for (int j = 0; j < C::kXTiles; ++j)
                        copy_scales(sfb + 4 * j, scale_desc(sc + (1 + j) * mx::kTileBytes));
                    const uint32_t sw = smem_u32(smem + size_t(s) * C::kStage), sx = sw + kWBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_mx(d, smem_desc_sw128(sw + kk * 32, 16, 1024), smem_desc_sw128(sx + kk * 32, 16, 1024),
                                idesc_mx(BN, kk), sfa, sfb, (k > 0 || kk > 0) ? 1u : 0u);
                    umma_commit(&empty[s]);
                    if (++s == uint32_t(C::kStages)) s = 0, phase ^= 1u;
                }
                if (!ok) break;
                umma_commit(&t_full[acc]);
                if (++acc == uint32_t(C::kAccs)) acc = 0, acc_phase ^= 1u;
            }
            umma_commit(drain);  // every MMA completes before tensor memory is released
            mbar_wait(drain, 0, &no_abort, kDrainTimeoutNs);
        }
    } else if (warp >= 6) {
        // ---------------- converters ----------------
        // A lane takes 16 packed bytes (32 values) of a row and stores them as two
        // 16-byte pieces with 8 bytes of codes each.  Both rings use the 128-byte swizzle
        // (piece p of row r at p ^ (r & 7)).  Lanes 0-3 read four neighbouring pieces of
        // one row and lanes 4-7 those of the row four further, which the swizzle puts in
        // the other half of the banks.
        const int tid = threadIdx.x - 6 * 32;
        const int sub = lane & 3, row0 = (tid >> 5) * 8 + ((lane >> 2) & 1) * 4 + (lane >> 3);
        uint32_t ps = 0, p_phase = 0, s = 0, phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            for (int k = 0; k < a.k_tiles && ok; k += 2) {
                ok = mbar_wait(&p_full[ps], p_phase, abort_flag, a.timeout_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const uint8_t* src = packed + size_t(ps) * kPackedBytes;
                for (int h = 0; h < 2 && k + h < a.k_tiles; ++h) {
                    ok = mbar_wait(&empty[s], phase ^ 1u, abort_flag, a.timeout_ns);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + size_t(s) * C::kStage;
#pragma unroll
                    for (int i = 0; i < kRows / 32; ++i) {
                        const int row = row0 + i * 32, x = row & 7;
                        const uint4 q = *reinterpret_cast<const uint4*>(src + row * 128 + (((4 * h + sub) ^ x) << 4));
                        *reinterpret_cast<uint2*>(dst + row * 128 + (((2 * sub) ^ x) << 4)) = make_uint2(q.x, q.y);
                        *reinterpret_cast<uint2*>(dst + row * 128 + (((2 * sub + 1) ^ x) << 4)) = make_uint2(q.z, q.w);
                    }
                    reinterpret_cast<uint32_t*>(scales + size_t(s) * C::kScales)[tid] =
                        reinterpret_cast<const uint32_t*>(packed_scales + (size_t(ps) * 2 + h) * mx::kTileBytes)[tid];
                    fence_async_shared();  // the tensor core reads these through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&w_full[s]);
                    if (++s == uint32_t(C::kStages)) s = 0, phase ^= 1u;
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_empty[ps]);
                if (++ps == uint32_t(C::kPacked)) ps = 0, p_phase ^= 1u;
            }
        }
    } else {
        // ---------------- epilogue: one vocabulary entry per lane ----------------
        const int q = warp & 3;
        uint32_t acc = 0, acc_phase = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const bool ok = mbar_wait(&t_full[acc], acc_phase, abort_flag, a.timeout_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int64_t v = int64_t(t / a.tiles_n) * kRows + q * 32 + lane;
            const int64_t n0 = int64_t(t % a.tiles_n) * BN;
            Out* out = static_cast<Out*>(a.out) + n0 * a.out_stride + v;
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + (uint32_t(q * 32) << 16) + acc * BN + c, r);
                tmem_ld_wait();
                const int left = int(a.n - n0 - c < 32 ? a.n - n0 - c : 32);
                const int width = BN < 32 ? (left < BN ? left : BN) : left;
                if (v < a.v) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < width && VCE_BOUNDS(n0 + c + j < a.n && v >= 0, a.dev_status))
                            store_logit(out + int64_t(c + j) * a.out_stride, __uint_as_float(r[j]));
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
    if (!byte_map(&tm_w, wc, cols / 2, uint64_t(a.v), kRows) || !byte_map(&tm_x, xc, cols, uint64_t(a.n), BN))
        return VCE_ERR_CUDA;
    a.tiles_v = int((a.v + kRows - 1) / kRows);
    a.tiles_n = int((a.n + BN - 1) / BN);
    const int64_t tiles = int64_t(a.tiles_v) * a.tiles_n;
    if (tiles > 0x7fffffff) return VCE_ERR_INVALID_ARG;
    count_launch();
    mx_linear_kernel<BN, Out><<<unsigned(tiles < dev.num_sms ? tiles : dev.num_sms), kThreads, Cfg<BN>::kSmem, s>>>(
        tm_w, tm_x, a);
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

template <typename Out>
vce_status dispatch(const void* xc, const void* wc, const LinearArgs& a, cudaStream_t s, const DeviceInfo& dev) {
    if (a.n <= 16) return launch<16, Out>(xc, wc, a, s, dev);
    if (a.n <= 32) return launch<32, Out>(xc, wc, a, s, dev);
    if (a.n <= 64) return launch<64, Out>(xc, wc, a, s, dev);
    if (a.n <= 128) return launch<128, Out>(xc, wc, a, s, dev);
    return launch<256, Out>(xc, wc, a, s, dev);
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
    a.x_scale_rows = mx::padded(n) / mx::kRowTile;
    a.out = out; a.out_stride = out_stride; a.dev_status = dev_status; a.timeout_ns = kPipeTimeoutNs;
    return out_dtype == VCE_BF16 ? dispatch<__nv_bfloat16>(x_codes, w_codes, a, s, dev)
                                 : dispatch<float>(x_codes, w_codes, a, s, dev);
}

}  // namespace vce
