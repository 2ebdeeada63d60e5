// Reordering of the beams' states: dst[b, k] = src[b, parent[b, k]] for every state, in place
// or into other buffers, as far as each request's positions are filled.
//
// Nothing but bytes moves, so the memory bounds it.  In place, without a second set of buffers:
// a thread takes one column of up to 16 bytes of a request's beams, reads it from every beam
// that is asked for before it writes any, and no other thread touches the column.  Beams that
// stay are neither read nor written (unless they are read for others).
//
// A block computes how much there is to do for each request of a state (columns of its filled
// positions, none where no beam moves), and its warps take their shares of all of that: requests of any
// lengths are spread evenly.  (Shares of a block each leave most threads idle where a part has few
// columns: 53 x 11 beams of 17 heads, 2 positions of 192 bytes each, 35 us instead of 14.)
//
// 8 caches of 256 x 8 x 1024 x 128 BF16, half filled on average, four of eight beams replaced by others of the
// same request, some of which are read for several: 283 us for 1.8 GB (6.4 TB/s).  24 x 5 beams of odd FP32 caches
// into other buffers: 60 us (6.7 TB/s).

#include "head_internal.cuh"

#include <algorithm>

namespace vce {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroup = 256;       // requests that a block looks after
constexpr int kStates = 128;      // states per launch
constexpr int kMaxBeams = VCE_BEAM_MAX_BEAMS;

struct State {
    const char* src;
    char* dst;
    int64_t src_stride, dst_stride, src_part, dst_part;  // bytes
    int64_t parts, run;        // runs of ``run`` bytes per row,
    int64_t positions, each;   // of positions of ``each`` bytes
    int width;                 // bytes of a column
};

struct ReorderArgs {
    const int64_t* parent;
    const int* lengths;
    int64_t batch;
    int beams, states;
    int* dev_status;
    State state[kStates];
};

struct Shared {
    int64_t before[kGroup + 1];  // units of the requests before
    int64_t columns[kGroup];
    int64_t warp_sum[kWarps];
    uint8_t n[kGroup];           // beams that move
    uint8_t to[kGroup][kMaxBeams], from[kGroup][kMaxBeams];
};

// U columns of each lane, from column ``c0`` on: of kMany beams at most.
template <typename V, int kMany, int U>
__device__ __forceinline__ void move(const State& st, const char* src, char* dst, int64_t c0, int64_t columns, int n,
                                     const uint8_t* to, const uint8_t* from) {
    V v[kMany][U];
    const int64_t c = c0 + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < kMany; ++j) {
        if (j >= n) break;
        const char* const at = src + from[j] * st.src_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * 32 < columns) v[j][u] = *reinterpret_cast<const V*>(at + (c + u * 32) * int64_t(sizeof(V)));
    }
#pragma unroll
    for (int j = 0; j < kMany; ++j) {
        if (j >= n) break;
        char* const at = dst + to[j] * st.dst_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * 32 < columns) *reinterpret_cast<V*>(at + (c + u * 32) * int64_t(sizeof(V))) = v[j][u];
    }
}

// Eight vectors per thread on their way at least, and registers held to what lets five blocks share an SM
// (a few addresses spill): 4.3 GB of caches in place took 375 us with the compiler's 126 registers, 293 with 48.
template <int kMany>
constexpr int columns_per_thread() { return kMany >= 8 ? 1 : 8 / kMany; }
template <int kMany>
constexpr int blocks_of() { return kMany <= 8 ? 5 : kMany == 16 ? 2 : 1; }  // per SM

template <int kMany>
__global__ void __launch_bounds__(kThreads, blocks_of<kMany>()) beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
    __shared__ Shared sh;
    constexpr int U = columns_per_thread<kMany>();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const State& st = a.state[blockIdx.y];
    const int64_t b0 = int64_t(blockIdx.z) * kGroup;
    const int group = int(min(int64_t(kGroup), a.batch - b0));
    const bool in_place = st.src == st.dst;

    int64_t units = 0;
    if (tid < group) {
        int n = 0;
        for (int k = 0; k < a.beams; ++k) {
            int64_t p = a.parent[(b0 + tid) * a.beams + k];
            if (p < 0 || p >= a.beams) {
                report(a.dev_status, VCE_DEVSTATUS_BAD_INDEX);
                p = k;
            }
            if (in_place && p == k) continue;
            sh.to[tid][n] = uint8_t(k), sh.from[tid][n] = uint8_t(p);
            ++n;
        }
        int64_t bytes = st.run;
        if (a.lengths) bytes = min(st.positions, max(int64_t(a.lengths[b0 + tid]), int64_t(0))) * st.each;
        const int64_t columns = bytes / st.width;
        sh.n[tid] = uint8_t(n), sh.columns[tid] = columns;
        if (n) units = (columns + U * 32 - 1) / (U * 32) * st.parts;
    }
    int64_t t = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += x;
    }
    if (lane == 31) sh.warp_sum[warp] = t;
    __syncthreads();
    for (int w = 0; w < warp; ++w) t += sh.warp_sum[w];
    sh.before[tid + 1] = t;
    if (tid == 0) sh.before[0] = 0;
    __syncthreads();

    const int64_t total = sh.before[kGroup];
    // (the shuffle tells the compiler that the unit is the warp's: addresses stay in uniform registers, 290 us against 590)
    for (int64_t unit = int64_t(blockIdx.x) * kWarps + __shfl_sync(0xffffffffu, warp, 0); unit < total; unit += int64_t(gridDim.x) * kWarps) {
        int r = 0;  // the last request with before[r] <= unit
#pragma unroll
        for (int step = kGroup / 2; step > 0; step >>= 1)
            if (sh.before[r + step] <= unit) r += step;
        const int64_t columns = sh.columns[r], i = unit - sh.before[r];
        const int64_t chunks = (columns + U * 32 - 1) / (U * 32);
        const int64_t part = i / chunks, c0 = (i - part * chunks) * (U * 32);
        const int64_t row = (b0 + r) * a.beams;
        const char* const src = st.src + row * st.src_stride + part * st.src_part;
        char* const dst = st.dst + row * st.dst_stride + part * st.dst_part;
        if (!VCE_BOUNDS(part < st.parts && columns * st.width <= st.run && c0 < columns, a.dev_status)) continue;
        switch (st.width) {
            case 16: move<uint4, kMany, U>(st, src, dst, c0, columns, sh.n[r], sh.to[r], sh.from[r]); break;
            case 8: move<uint64_t, kMany, U>(st, src, dst, c0, columns, sh.n[r], sh.to[r], sh.from[r]); break;
            case 4: move<uint32_t, kMany, U>(st, src, dst, c0, columns, sh.n[r], sh.to[r], sh.from[r]); break;
            case 2: move<uint16_t, kMany, U>(st, src, dst, c0, columns, sh.n[r], sh.to[r], sh.from[r]); break;
            default: move<uint8_t, kMany, U>(st, src, dst, c0, columns, sh.n[r], sh.to[r], sh.from[r]); break;
        }
    }
}

// The widest column that divides everything.
int column_width(const vce_state& s, bool by_length) {
    uint64_t all = uint64_t(reinterpret_cast<uintptr_t>(s.src)) | uint64_t(reinterpret_cast<uintptr_t>(s.dst)) |
                   uint64_t(s.src_row_stride) | uint64_t(s.dst_row_stride) | 16;
    if (s.parts > 1) all |= uint64_t(s.src_part_stride) | uint64_t(s.dst_part_stride);
    all |= by_length ? uint64_t(s.position_bytes) : uint64_t(s.positions) * uint64_t(s.position_bytes);
    return int(all & (~all + 1));
}

}  // namespace

vce_status launch_beam_reorder(const vce_state* states, int count, const int64_t* parent, int64_t batch, int beams,
                               const int* lengths, int* dev_status, cudaStream_t s, const DeviceInfo& dev) {
    if (batch == 0) return VCE_OK;
    const int many = beams <= 4 ? 4 : beams <= 8 ? 8 : beams <= 16 ? 16 : 32;
    const int per_unit = (many >= 8 ? 1 : 8 / many) * 32;
    auto kernel = many == 4 ? beam_reorder_kernel<4> : many == 8 ? beam_reorder_kernel<8>
                : many == 16 ? beam_reorder_kernel<16> : beam_reorder_kernel<32>;
    const int64_t groups = (batch + kGroup - 1) / kGroup;
    ReorderArgs a;
    a.parent = parent, a.lengths = lengths, a.batch = batch, a.beams = beams, a.dev_status = dev_status;
    for (int i = 0; i < count;) {
        a.states = 0;
        int64_t most = 1;  // blocks for a group of requests, at full length
        for (; i < count && a.states < kStates; ++i) {
            const vce_state& x = states[i];
            if (x.parts == 0 || x.positions == 0 || x.position_bytes == 0) continue;
            State& st = a.state[a.states++];
            st = {static_cast<const char*>(x.src), static_cast<char*>(x.dst), x.src_row_stride, x.dst_row_stride,
                  x.src_part_stride, x.dst_part_stride, x.parts, x.positions * x.position_bytes, x.positions, x.position_bytes,
                  column_width(x, lengths != nullptr)};
            const int64_t units = (st.run / st.width + per_unit - 1) / per_unit * st.parts * std::min<int64_t>(batch, kGroup);
            most = std::max(most, (units + kWarps - 1) / kWarps);
        }
        if (a.states == 0) break;
        // As many blocks as run at once, shared by the states; twice as many where there are many units, so
        // that the ends even out (293 -> 290 us; caches of a few positions 6.5 -> 8.1).
        int64_t share = std::max<int64_t>(1, int64_t(dev.num_sms) * 5 / (a.states * groups));
        if (most >= 8 * share) share *= 2;
        count_launch();
        kernel<<<dim3(unsigned(std::min(most, share)), unsigned(a.states), unsigned(groups)), kThreads, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return VCE_ERR_CUDA;
    }
    return VCE_OK;
}

}  // namespace vce
