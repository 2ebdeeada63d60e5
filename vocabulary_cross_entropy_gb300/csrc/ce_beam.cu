// The next hypotheses of a beam search from the logits of all beams.
//
// With m the largest logit of a row and S = sum exp(z - m), token v takes the beam's score s
// to s + (z_v - m) - ln S.  Of all tokens of a request's beams the best few are wanted, in
// order.  Two kernels: one finds each row's S and its best tokens, the other, one warp per
// request, merges the beams' lists.
//
// Rows are compared with one another, so S has to be good to far more than FP32's 2^-24: two
// candidates of different beams 10^-7 apart would change places.  And equal rows have to give
// equal S bit for bit, as the lowest beam comes first among equals.  Therefore
//   - the tokens at or above a bound (a little more than the wanted ones, and the bulk of
//     a peaked row's mass) enter S as whole numbers, good to 2^-36 (token_order.cuh);
//   - of the others each weight is an FP32 exponential; a thread adds up its own few, by
//     a division of the row that goes by the index of the token alone, never by the address,
//     and the threads' sums are joined as whole numbers, in any order.
//
// A row is shared by a cluster of blocks such that a block's part fits its registers: the row
// is read once, its maximum and the bound are found, and the sum and the survivors come from
// the registers.  The bound is the j-th largest of the maxima of disjoint groups of a block's
// elements, j = the wanted number over the blocks; the least of the blocks' bounds is at
// most the wanted number's largest.

#include "head_internal.cuh"
#include "sm100_ptx.cuh"
#include "token_order.cuh"

#include <math.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kHold = 8;              // vectors that a thread holds
constexpr int kCap = 1024;            // collected keys
constexpr int kMaxCluster = 8;
constexpr int kMaxCount = VCE_BEAM_MAX_COUNT;
constexpr int kMaxBeams = VCE_BEAM_MAX_BEAMS;

// What the first kernel leaves of a row, in front of its keys.
struct RowHead {
    float m;
    int n;          // keys
    uint64_t mass;  // S in units of 2^-Q
};

struct RowArgs {
    const void* logits;
    int64_t stride;
    int vocab;
    const float* score;
    const uint8_t* ended;
    int count, cluster;
    int q_bits;        // Q
    float least_log2;  // weights below it count as 0
    RowHead* heads;
    uint64_t* keys;
    int* dev_status;
};

struct Shared {
    uint64_t list[kCap];
    uint64_t tmp[kThreads / 2];
    uint64_t table[kSteps];
    uint64_t join[kMaxCluster * kMaxCount];  // block 0's: the blocks' keys, and below their numbers and masses
    uint64_t part_mass[kMaxCluster];
    uint32_t part_n[kMaxCluster];
    float row_max[kMaxCluster], bound[kMaxCluster];  // put by every block into every block
    uint64_t mass;
    float group[kThreads];
    float warp_max[kWarps];
    float my_bound;
    uint32_t n_list;
};

__device__ __forceinline__ void put(uint64_t* p, int rank, uint64_t v) {
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), uint32_t(rank))), "l"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t* p, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), uint32_t(rank))), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {  // of two BF16 each
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest of a vector's elements; a NaN stays.
template <typename T>
__device__ __forceinline__ float vector_max(uint4 v) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = max2_nan(max2_nan(v.x, v.y), max2_nan(v.z, v.w));
        return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return max_nan(max_nan(element<T>(v, 0), element<T>(v, 1)), max_nan(element<T>(v, 2), element<T>(v, 3)));
    }
}

// A block's part of a row.  Group g is the elements [g VE, (g + 1) VE), whatever their address:
// where the row starts off a 16-byte boundary a group is cut out of two vectors.  The groups of
// which both lie in the row for any address, [1, vocab / VE - 1), are divided among the blocks,
// [g0, g1) to this one; the elements before and behind them, at most 4 VE, go one to a thread
// of the last block.
template <typename T>
struct Part {
    static constexpr int VE = 16 / int(sizeof(T));
    const T* row;
    int off, vocab;
    int g0, g1;
    bool last;
    int* dev_status;

    __device__ __forceinline__ uint4 load(int g, int skip) const {  // vector g + skip of the aligned ones
        const T* at = row + (int64_t(g + skip) * VE - off);
        if (VCE_BOUNDS(aligned16(at) && at >= row && at + VE <= row + vocab, dev_status))
            return __ldg(reinterpret_cast<const uint4*>(at));
        return nothing();
    }
    __device__ static __forceinline__ uint4 nothing() {
        const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
        return make_uint4(w, w, w, w);
    }
    // Elements ``off`` .. of two neighbouring vectors.
    __device__ __forceinline__ uint4 cut(uint4 a, uint4 b) const {
        const int bytes = off * int(sizeof(T));
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (bytes & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (bytes & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const int bits = (bytes & 3) * 8;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
    // Groups g0 + chunk kHold kThreads + tid + k kThreads of the part, -inf past its end.
    __device__ __forceinline__ void fetch(uint4 (&v)[kHold], int chunk) const {
        const int g = g0 + chunk * (kHold * kThreads) + int(threadIdx.x);
        if (off == 0) {
#pragma unroll
            for (int k = 0; k < kHold; ++k) v[k] = g + k * kThreads < g1 ? load(g + k * kThreads, 0) : nothing();
        } else {
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                v[k] = nothing();
                if (g + k * kThreads < g1) v[k] = cut(load(g + k * kThreads, 0), load(g + k * kThreads, 1));
            }
        }
    }
    __device__ __forceinline__ int chunks() const { return max(1, (g1 - g0 + kHold * kThreads - 1) / (kHold * kThreads)); }
    // The index of this thread's single element, or -1.
    __device__ __forceinline__ int single() const {
        if (!last) return -1;
        const int first = min(VE, vocab), tail = max(vocab / VE - 1, 1) * VE, t = int(threadIdx.x);
        return t < first ? t : tail + t - first < vocab ? tail + t - first : -1;
    }
    __device__ __forceinline__ float single_value(int i) const {
        return i >= 0 && VCE_BOUNDS(i < vocab, dev_status) ? one(row + i) : -INFINITY;
    }
};

__device__ __forceinline__ uint64_t heavy_weight(const Scale& sc, float z, const RowArgs& a, const uint64_t* table) {
    return log2_weight(sc, z) > a.least_log2 ? weight_of(sc, z, table, a.q_bits) : 0;
}

__device__ __forceinline__ void add_mass(uint64_t* at, uint64_t w) {
    atomicAdd(reinterpret_cast<unsigned long long*>(at), static_cast<unsigned long long>(w));
}

// A block with more elements at or above the bound than the list holds (equal logits, or a
// few groups that have them all): element by element, the best ``count`` so far are kept
// whenever the list fills.  Their weights all enter the mass.  Rare, and kept out of the
// common code.
template <typename T>
__device__ __noinline__ void collect_many(const RowArgs& a, Shared& sh, const Part<T>& part, const Scale& sc, float bound) {
    constexpr int VE = Part<T>::VE;
    __syncthreads();
    if (threadIdx.x == 0) sh.n_list = 0;
    __syncthreads();
    uint64_t least = 0, mass = 0;
    auto take = [&](float z, int i) {
        if (z >= bound && z > -INFINITY) {
            mass += heavy_weight(sc, z, a, sh.table);
            const uint64_t key = key_of(z, i);
            if (key > least) sh.list[atomicAdd(&sh.n_list, 1u)] = key;  // never full here: see below
        }
        __syncthreads();
        const uint32_t n = sh.n_list;
        __syncthreads();
        if (n > kCap - kThreads) {
            sort_list<kThreads>(sh.list, int(n), sh.tmp);
            if (threadIdx.x == 0) sh.n_list = uint32_t(a.count);
            least = sh.list[a.count - 1];
            __syncthreads();
        }
    };
    const int single = part.single();
    take(part.single_value(single), single);
    for (int c = 0; c < part.chunks(); ++c) {
        uint4 v[kHold];
        part.fetch(v, c);
        const int g = part.g0 + c * (kHold * kThreads) + int(threadIdx.x);
#pragma unroll 1
        for (int k = 0; k < kHold; ++k) {
            if (part.g0 + (c * kHold + k) * kThreads >= part.g1) break;
#pragma unroll 1
            for (int e = 0; e < VE; ++e) {
                uint4 x = v[0];
#pragma unroll
                for (int j = 1; j < kHold; ++j) x = j == k ? v[j] : x;
                take(element<T>(x, e), (g + k * kThreads) * VE + e);
            }
        }
    }
    add_mass(&sh.mass, mass);
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) ce_beam_rows(const RowArgs a) {
    __shared__ Shared sh;
    constexpr int VE = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int rank = a.cluster == 1 ? 0 : int(cluster_ctarank());
    const int64_t row = int64_t(blockIdx.x) / a.cluster;
    RowHead* const head = a.heads + row;
    const float score = a.score[row];
    if (score == -INFINITY || (a.ended && a.ended[row])) return;  // nothing to read: the merge knows
    if (a.cluster > 1) cluster_arrive();  // waited for below, before the first store to another block

    Part<T> part;
    part.row = static_cast<const T*>(a.logits) + row * a.stride;
    part.off = int(reinterpret_cast<uintptr_t>(part.row) / sizeof(T) % VE);
    part.vocab = a.vocab;
    const int end = max(a.vocab / VE - 1, 1), per = (end - 1 + a.cluster - 1) / a.cluster;
    part.g0 = 1 + rank * per, part.g1 = min(end, 1 + (rank + 1) * per);
    part.last = rank == a.cluster - 1;
    part.dev_status = a.dev_status;

    // ---- the largest logit, and the largest of every thread's elements ----
    const int single = part.single();
    const float z1 = part.single_value(single);
    const int chunks = part.chunks();
    float m = z1;
    uint4 v[kHold];
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {  // the last chunk stays
        part.fetch(v, c);
        if constexpr (sizeof(T) == 2) {
            uint32_t w = 0xff80ff80u;
#pragma unroll
            for (int k = 0; k < kHold; ++k) w = max2_nan(w, max2_nan(max2_nan(v[k].x, v[k].y), max2_nan(v[k].z, v[k].w)));
            m = max_nan(m, max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
        } else {
#pragma unroll
            for (int k = 0; k < kHold; ++k) m = max_nan(m, vector_max<T>(v[k]));
        }
    }
    sh.group[tid] = m;
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = max_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    if ((tid & 31) == 0) sh.warp_max[tid >> 5] = wm;
    if (tid < kSteps) sh.table[tid] = kExp2Table[tid];
    if (tid == 0) sh.my_bound = -INFINITY, sh.n_list = 0, sh.mass = 0;
    __syncthreads();
    {
        const int j = (a.count + a.cluster - 1) / a.cluster;
        int groups = 64;  // of neighbouring threads: larger groups bound less tightly but rank faster
        while (groups < 2 * j) groups *= 2;
        const int width = kThreads / groups;
        float g = -INFINITY;
        if (tid < groups)
            for (int i = 0; i < width; ++i) g = fmaxf(g, sh.group[tid * width + i]);
        __syncthreads();
        if (tid < groups) sh.group[tid] = g;
        __syncthreads();
        if (tid < groups) {
            int before = 0;
#pragma unroll 8
            for (int i = 0; i < groups; ++i) before += sh.group[i] > g || (sh.group[i] == g && i < tid);
            if (before == j - 1) sh.my_bound = g;
        }
        __syncthreads();
    }
    if (a.cluster > 1) cluster_wait();  // every block of the cluster runs: its shared memory may be written
    if (tid < a.cluster) {
        float r = sh.warp_max[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) r = max_nan(r, sh.warp_max[w]);
        if (a.cluster == 1) {
            sh.row_max[0] = r, sh.bound[0] = sh.my_bound;
        } else {
            put(reinterpret_cast<uint32_t*>(&sh.row_max[rank]), tid, __float_as_uint(r));
            put(reinterpret_cast<uint32_t*>(&sh.bound[rank]), tid, __float_as_uint(sh.my_bound));
        }
    }
    if (a.cluster == 1) __syncthreads();
    else cluster_sync();
    float row_max = -INFINITY, bound = INFINITY;
    for (int c = 0; c < a.cluster; ++c) {
        row_max = max_nan(row_max, sh.row_max[c]);
        bound = fminf(bound, sh.bound[c]);
    }
    if (!(row_max < INFINITY) || row_max == -INFINITY || !(score < INFINITY)) {  // the same in every block
        if (rank == 0 && tid == 0) {
            *head = {0.f, 0, 0};
            report(a.dev_status, VCE_DEVSTATUS_BAD_ROW);
        }
        return;
    }

    // ---- the sum of the weights below the bound; the keys of the elements at or above it ----
    const Scale sc = make_scale(row_max, 1.f);
    float2 sum[4] = {};
    auto heavy = [&](float z, int i) {  // whether z is; if so its key is collected
        if (!(z >= bound && z > -INFINITY)) return false;
        const uint32_t at = atomicAdd(&sh.n_list, 1u);
        if (at < uint32_t(kCap)) sh.list[at] = key_of(z, i);
        return true;
    };
    const float2 minus = make_float2(-row_max, -row_max), log2e = make_float2(kLog2e, kLog2e);
#pragma unroll 1
    for (int c = chunks - 1; c >= 0; --c) {
        if (c != chunks - 1) part.fetch(v, c);
        const int g = part.g0 + c * (kHold * kThreads) + tid;
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            float z[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) z[e] = element<T>(v[k], e);
            if (vector_max<T>(v[k]) >= bound) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (heavy(z[e], (g + k * kThreads) * VE + e)) z[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                const float2 x = __fmul2_rn(__fadd2_rn(make_float2(z[e], z[e + 1]), minus), log2e);
                sum[e / 2] = __fadd2_rn(sum[e / 2], make_float2(ex2f(x.x), ex2f(x.y)));
            }
        }
    }
    if (!heavy(z1, single)) sum[0].x += ex2f((z1 - row_max) * kLog2e);
    {
        const float2 s = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
        uint64_t w = __float2ull_rn(ldexpf(s.x + s.y, a.q_bits));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        if ((tid & 31) == 0) add_mass(&sh.mass, w);
    }
    __syncthreads();
    uint32_t n = sh.n_list;
    if (n > uint32_t(kCap)) {
        collect_many(a, sh, part, sc, bound);
        n = sh.n_list;
    } else {
        for (uint32_t i = tid; i < n; i += kThreads) add_mass(&sh.mass, heavy_weight(sc, key_logit(sh.list[i]), a, sh.table));
    }
    if (a.cluster > 1) {
        if (n > uint32_t(kMaxCount)) {
            sort_list<kThreads>(sh.list, int(n), sh.tmp);
            n = min(n, uint32_t(a.count));
        }
        __syncthreads();  // the mass
        if (uint32_t(tid) < n) put(&sh.join[rank * kMaxCount + tid], 0, sh.list[tid]);
        if (tid == 0) {
            put(&sh.part_n[rank], 0, n);
            put(&sh.part_mass[rank], 0, sh.mass);
        }
        cluster_sync();
        if (rank != 0) return;
        uint32_t total = 0;
        uint64_t mass = 0;
        for (int c = 0; c < a.cluster; ++c) {
            const uint32_t part_n = sh.part_n[c];
            if (uint32_t(tid) < part_n) sh.list[total + tid] = sh.join[c * kMaxCount + tid];
            total += part_n;
            mass += sh.part_mass[c];
        }
        n = total;
        __syncthreads();
        if (tid == 0) sh.mass = mass;
    }
    __syncthreads();
    sort_list<kThreads>(sh.list, int(n), sh.tmp);
    n = min(n, uint32_t(a.count));
    if (uint32_t(tid) < n) a.keys[row * a.count + tid] = sh.list[tid];
    if (tid == 0) *head = {row_max, int(n), sh.mass};
}

// ---------------------------------------------------------------------------
// the merge
// ---------------------------------------------------------------------------

struct MergeArgs {
    int64_t batch;
    int beams, count, end, keep, q_bits;
    float penalty;
    const RowHead* heads;
    const uint64_t* keys;
    const float* score;
    const uint8_t* ended;
    const int* length;
    int64_t *token, *parent;
    float* out_score;
    uint8_t* out_ended;
    int* out_length;
    int* dev_status;
};

__device__ __forceinline__ uint64_t order_bits(double z) {  // monotone in z; -0 counts as 0
    const uint64_t b = uint64_t(__double_as_longlong(z + 0.0));
    return b ^ (uint64_t(int64_t(b) >> 63) | 0x8000000000000000ull);
}

// One warp per request; lane k holds beam k's best candidate that has not been taken.
__global__ void __launch_bounds__(32) ce_beam_merge(const MergeArgs a) {
    extern __shared__ uint64_t keys[];  // beams x count, then what was chosen
    const int lane = threadIdx.x;
    const int64_t request = blockIdx.x, row = request * a.beams + lane;
    const bool mine = lane < a.beams;
    double* const chosen = reinterpret_cast<double*>(keys + a.beams * a.count);
    int* const chosen_token = reinterpret_cast<int*>(chosen + a.count);
    int* const chosen_parent = chosen_token + a.count;
    int* const place = chosen_parent + a.count;

    cudaGridDependencySynchronize();
    float score = -INFINITY;
    int length = 0, n = 0;
    bool ended = false;
    RowHead head{0.f, 0, 0};
    if (mine) {
        score = a.score[row];
        ended = a.ended && a.ended[row];
        length = a.length ? a.length[row] : 0;
        if (ended) {
            n = score > -INFINITY && score < INFINITY;
            if (!n && score != -INFINITY) report(a.dev_status, VCE_DEVSTATUS_BAD_ROW);
        } else if (score != -INFINITY) {
            head = a.heads[row];
            n = head.n;
        }
    }
    for (int i = lane; i < a.beams * a.count; i += 32) {
        const int k = i / a.count;
        const int nk = k < a.beams ? a.count : 0;
        if (nk) keys[i] = a.keys[request * a.beams * a.count + i];  // those past a row's number are not looked at
    }
    __syncwarp();

    const double log_s = head.n ? log(ldexp(double(head.mass), -a.q_bits)) : 0.0;
    const int after = ended ? length : length + 1;
    const double norm = a.penalty != 0.f ? pow(double(max(after, 1)), double(a.penalty)) : 1.0;
    int at = 0, token = -1;
    double total = 0.0;
    uint64_t value = 0;  // order of the candidate's value; 0: none
    auto next = [&]() {
        value = 0;
        if (at >= n) return;
        if (ended) {
            token = a.end, total = double(score);
        } else {
            const uint64_t key = keys[lane * a.count + at];
            token = key_index(key);
            total = double(score) + ((double(key_logit(key)) - double(head.m)) - log_s);
        }
        value = order_bits(a.penalty != 0.f ? total / norm : total);
        ++at;
    };
    next();
    uint32_t taken = 0;
    uint64_t deferred = 0;  // chosen ones without a place of their own
    for (int i = 0; i < a.count; ++i) {
        const uint32_t high = __reduce_max_sync(0xffffffffu, uint32_t(value >> 32));
        const uint32_t low = __reduce_max_sync(0xffffffffu, uint32_t(value >> 32) == high ? uint32_t(value) : 0u);
        const bool none = (high | low) == 0;
        const int best = __ffs(int(__ballot_sync(0xffffffffu, value == (uint64_t(high) << 32 | low)))) - 1;
        if (none) {
            if (lane == 0) chosen_parent[i] = -1;
            deferred |= uint64_t(1) << i;
        } else {
            const bool first = !(taken >> best & 1);
            taken |= 1u << best;
            if (!first) deferred |= uint64_t(1) << i;
            if (lane == best) {
                chosen[i] = total, chosen_token[i] = token, chosen_parent[i] = lane, place[i] = lane;
                next();
            }
        }
        __syncwarp();
    }
    if (a.keep) {
        uint32_t free = ~taken;
        for (int i = 0; i < a.count; ++i)
            if (deferred >> i & 1) {
                if (lane == 0) place[i] = __ffs(int(free)) - 1;
                free &= free - 1;
            }
        __syncwarp();
    }
    for (int i0 = 0; i0 < a.count; i0 += 32) {
        const int i = i0 + lane;
        const bool valid = i < a.count && chosen_parent[i] >= 0;
        const int to = i >= a.count ? 0 : a.keep ? place[i] : i;
        const int parent = valid ? chosen_parent[i] : to % a.beams;
        const int was_length = __shfl_sync(0xffffffffu, length, parent);
        const bool was_ended = __shfl_sync(0xffffffffu, int(ended), parent);
        if (i >= a.count) continue;
        const int64_t out = request * a.count + to;
        const int tok = valid ? chosen_token[i] : -1;
        a.token[out] = tok;
        a.parent[out] = parent;
        a.out_score[out] = valid ? float(chosen[i]) : -INFINITY;
        if (a.out_ended) a.out_ended[out] = valid && (was_ended || tok == a.end);
        if (a.out_length) a.out_length[out] = was_length + (valid && !was_ended);
    }
}

}  // namespace

size_t ce_beam_ws_bytes(int64_t rows, int count) {
    return align256(size_t(rows) * sizeof(RowHead)) + size_t(rows) * size_t(count) * sizeof(uint64_t);
}

vce_status launch_ce_beam(const void* logits, int dtype, int64_t batch, int beams, int64_t vocab, int64_t stride,
                          const float* score, const uint8_t* ended, const int* length, int64_t end, float penalty,
                          int count, int keep, int64_t* token, int64_t* parent, float* out_score,
                          uint8_t* out_ended, int* out_length, void* ws, int* dev_status, cudaStream_t s,
                          const DeviceInfo& dev) {
    const int64_t rows = batch * beams;
    if (rows == 0) return VCE_OK;
    int bits = 0;
    while ((int64_t(1) << bits) < vocab) ++bits;
    RowArgs a{logits, stride, int(vocab), score, ended, count, 1, 63 - bits < 44 ? 63 - bits : 44, 0.f,
              static_cast<RowHead*>(ws),
              reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + align256(size_t(rows) * sizeof(RowHead))), dev_status};
    a.least_log2 = -float(a.q_bits + 1) + 0x1p-10f;
    // As many blocks per row as hold it in registers, and as fill the SMs where rows are few.
    const int64_t vectors = vocab / (dtype == VCE_BF16 ? 8 : 4);
    while (a.cluster < kMaxCluster &&
           (vectors > int64_t(a.cluster) * kHold * kThreads ||
            (rows * a.cluster * 2 <= 2 * dev.num_sms && vectors >= int64_t(a.cluster) * 2 * kThreads)))
        a.cluster *= 2;
    if (rows * a.cluster > 0x7fffffff) return VCE_ERR_INVALID_ARG;
    auto kernel = dtype == VCE_BF16 ? ce_beam_rows<__nv_bfloat16> : ce_beam_rows<float>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(rows * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(a.cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    count_launch();
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return VCE_ERR_CUDA;

    const MergeArgs g{batch, beams, count, int(end), keep, a.q_bits, penalty, a.heads, a.keys, score, ended, length,
                      token, parent, out_score, out_ended, out_length, dev_status};
    cudaLaunchConfig_t mcfg{};
    mcfg.gridDim = dim3(unsigned(batch));
    mcfg.blockDim = dim3(32);
    mcfg.dynamicSmemBytes = size_t(beams) * count * 8 + size_t(count) * 20;  // at most 18 KB
    mcfg.stream = s;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    mcfg.attrs = &early;
    mcfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&mcfg, ce_beam_merge, g) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
