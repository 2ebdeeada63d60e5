// The next hypotheses of a beam search from the logits of all beams.
//
// With m the largest logit of a row and S = sum exp(z - m), token v takes the beam's score s
// to s + (z_v - m) - ln S.  Of all tokens of a request's beams the best few are wanted, in
// order.  Two kernels: one finds the sums and the best tokens of parts of the rows, the other,
// a block per request, joins the parts and merges the beams.
//
// Rows are compared with one another, so S has to be good to more than FP32's 2^-24: two
// candidates of different beams 10^-7 apart would change places.  And equal rows have to give
// equal S bit for bit, as the lowest beam comes first among equals.  Therefore
//   - the tokens at or above a bound (a little more than the wanted ones, and the bulk of
//     a peaked row's mass) enter S as whole numbers, good to 2^-36 (token_order.cuh);
//   - of the others each weight is an FP32 exponential; a thread adds up its own few, by
//     a division of the row that goes by the index of the token alone, never by the address,
//     and the threads' sums are joined as whole numbers, in any order.
// What is wrong with ln S is mostly common to all rows: 3e-8 from the rounding of log2(e), 5e-9
// of it differing from row to row (128256 tokens).  The FP32 exponent is one FMA, z log2(e) - m log2(e), whose
// second term is rounded once for the row: 2^r, r the remainder of that rounding, multiplies the row's sum.
//
// A part is copied into a block's shared memory at once, asynchronously: its maximum and the bound
// are found, and the sum and the survivors come from there.  The bound is the n-th largest of
// the maxima of disjoint groups of the part's elements, n = the wanted number.  Only the few threads
// that have an element at or above it know; what they hold is looked through by all.  A
// further warp does what one warp does alone (it waits for the copy, finds the bound, sorts
// the survivors while the others add up the weights).
//
// What bounds it: the chain of a block's steps, of which five blocks per SM cover each other.
// 64 x 8 x 128256 BF16 (85% of the beams go on): 36 us and 7 for the merge, where the copies alone take
// 20 and the memory's rate allows 17.  Parts of 32 KB, 256 threads; 64 KB and 512: 37; 24 KB: 46.  With a
// row's parts in a cluster of blocks that agreed on a maximum and joined their lists 76 + 10, most of
// it waits at barriers; with the parts in registers, which take many more instructions and leave
// room for two blocks, 61 + 14; with each thread looking for its survivors by itself 59 + 8; with as many
// blocks as run at once, each taking one part after the other, 44 + 7 (uneven ends, and registers).

#include "head_internal.cuh"
#include "sm100_ptx.cuh"
#include "token_order.cuh"

#include <algorithm>
#include <climits>
#include <math.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kThreads = 256;         // that go through a part; a further warp serves them
constexpr int kWarps = kThreads / 32;
constexpr int kHold = 8;              // vectors of a part per thread
constexpr int kBlocks = 5;            // per SM
constexpr int kBytes = (kHold * kThreads + 1) * 16;  // one more where the row is off a 16-byte boundary
constexpr int kCap = 1024;            // collected keys
constexpr int kFew = 128;             // as many are sorted by a warp
constexpr int kMaxParts = 16;
constexpr int kMaxCount = VCE_BEAM_MAX_COUNT;
constexpr int kMaxBeams = VCE_BEAM_MAX_BEAMS;
constexpr int kRowWarps = 8;          // of the merge; one more takes logarithms meanwhile
constexpr int kMergeThreads = kRowWarps * 32 + 32;
constexpr int kMergeBytes = 200 << 10;  // of shared memory, at most

// What the first kernel leaves of a part of a row, beside its keys (descending).
struct PartHead {
    float m;
    int n;          // keys; -1: a NaN or +inf was found
    uint64_t mass;  // sum of exp(z - m) in units of 2^-Q
};

struct RowArgs {
    const void* logits;
    int64_t stride;
    int vocab;
    const float* score;
    const uint8_t* ended;
    int count, parts;
    int per;           // groups of a part
    int q_bits;        // Q
    float least_log2;  // weights below it count as 0
    PartHead* heads;
    uint64_t* keys;
    int* dev_status;
};

struct Shared {
    uint64_t list[kCap];
    uint64_t table[kSteps];
    uint64_t arrived;  // mbarrier of the part's copy
    uint64_t mass;     // of collected elements
    alignas(16) uint32_t group[128];
    float warp_sum[kWarps];
    uint16_t hot[kThreads];  // threads with collected elements
    float bound, top;
    uint32_t n_list, n_hot;
    int abort;
};

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {  // of two BF16 each
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A block's part of a row.  Group g is the elements [g VE, (g + 1) VE), whatever their address:
// where the row starts off a 16-byte boundary a group is cut out of two vectors.  The groups of
// which both lie in the row for any address, [1, vocab / VE - 1), are divided among the parts,
// [g0, g1) to this one; the elements before them go one to a thread of the first part, those
// behind, fewer than 3 VE, of the last.  So a part's tokens come before the next one's.
// The groups are copied to ``data`` a chunk of kHold kThreads at a time (parts of up to 32 KB have
// one chunk, which stays).  A BF16 thread takes whole groups; an FP32 thread elements that are
// kThreads apart, which it reads without cutting.
template <typename T>
struct Part {
    static constexpr int VE = 16 / int(sizeof(T));
    static constexpr int kChunk = kHold * kThreads;
    const T* row;
    uint4* data;
    Shared* sh;
    int off, vocab;
    int g0, g1;
    bool first, last;
    int* dev_status;
    uint32_t parity;
    int now;  // groups in data

    __device__ __forceinline__ int chunks() const { return max(1, (g1 - g0 + kChunk - 1) / kChunk); }
    __device__ __forceinline__ int groups(int c) const { return max(0, min(kChunk, g1 - g0 - c * kChunk)); }
    // Thread 0 starts the copy of a chunk; all threads wait for it.
    __device__ __forceinline__ void start(int c) const {
        const int n = groups(c);
        if (n == 0) return;
        const T* const at = row + (int64_t(g0 + c * kChunk) * VE - off);
        const uint32_t bytes = uint32_t(n + (off > 0)) * 16;
        mbar_arrive_expect_tx(&sh->arrived, bytes);
        if (VCE_BOUNDS(aligned16(at) && at >= row && at + bytes / sizeof(T) <= row + vocab && bytes <= kBytes, dev_status))
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         ::"r"(smem_u32(data)), "l"(at), "r"(bytes), "r"(smem_u32(&sh->arrived))
                         : "memory");
    }
    // All threads; the serving warp polls.  False when the copy did not arrive: the results are lost, which
    // the status tells.
    __device__ __forceinline__ bool wait(int c) {
        now = groups(c);
        if (now == 0) return true;
        const bool ok = threadIdx.x < kThreads || mbar_wait(&sh->arrived, parity, &sh->abort, kPipeTimeoutNs);
        parity ^= 1;
        return __syncthreads_and(ok);
    }
    __device__ __forceinline__ bool next(int c) {  // after every thread's last read of data
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // what threads wrote there comes before the copy
        __syncthreads();
        if (threadIdx.x == kThreads) start(c);
        return wait(c);
    }
    // Elements ``off`` .. of two neighbouring vectors (BF16).
    __device__ __forceinline__ uint4 cut(uint4 a, uint4 b) const {
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (off & 4) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (off & 2) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const int bits = (off & 1) * 16;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
    // fn of the chunk's vectors of this thread: every VE elements it takes; -inf past the end.
    template <typename F>
    __device__ __forceinline__ void each(F fn) const {
        const int tid = int(threadIdx.x), whole = now / kThreads;
        if constexpr (sizeof(T) == 2) {
            const uint4* const at = data + tid;
            if (off == 0) {
#pragma unroll 4
                for (int k = 0; k < whole; ++k) fn(at[k * kThreads]);
            } else {
#pragma unroll 2
                for (int k = 0; k < whole; ++k) fn(cut(at[k * kThreads], at[k * kThreads + 1]));
            }
            const int i = whole * kThreads;
            if (i + tid < now) fn(off == 0 ? at[i] : cut(at[i], at[i + 1]));
        } else {
            const uint32_t* const at = reinterpret_cast<const uint32_t*>(data) + off + tid;
#pragma unroll 4
            for (int k = 0; k < whole; ++k) {
                const uint32_t* const w = at + k * VE * kThreads;
                fn(make_uint4(w[0], w[kThreads], w[2 * kThreads], w[3 * kThreads]));
            }
            const int i = whole * VE * kThreads, n = now * VE - tid;
            if (i < n) {
                uint4 v = nothing();
                v.x = at[i];
                if (i + kThreads < n) v.y = at[i + kThreads];
                if (i + 2 * kThreads < n) v.z = at[i + 2 * kThreads];
                if (i + 3 * kThreads < n) v.w = at[i + 3 * kThreads];
                fn(v);
            }
        }
    }
    __device__ static __forceinline__ uint4 nothing() {
        const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
        return make_uint4(w, w, w, w);
    }
    // Thread t's j-th element of the chunk, j < kHold VE: its place among them, or -1.
    __device__ __forceinline__ int place(int t, int j) const {
        const int i = sizeof(T) == 2 ? (j / VE * kThreads + t) * VE + j % VE : j * kThreads + t;
        return i < now * VE ? i : -1;
    }
    __device__ __forceinline__ T* element_at(int i) const { return reinterpret_cast<T*>(data) + off + i; }
    __device__ __forceinline__ int token(int c, int i) const { return (g0 + c * kChunk) * VE + i; }
    // The index of this thread's single element, or -1.
    __device__ __forceinline__ int single() const {  // (the serving warp has none)
        if (threadIdx.x >= kThreads) return -1;
        const int t = int(threadIdx.x), head = first ? min(VE, vocab) : 0;
        const int i = t < head ? t : max(vocab / VE - 1, 1) * VE + t - head;
        return t < head || (last && i < vocab) ? i : -1;
    }
    __device__ __forceinline__ float single_value(int i) const {
        return i >= 0 && VCE_BOUNDS(i < vocab, dev_status) ? one(row + i) : -INFINITY;
    }
};

// 2^r for the remainder r of neg = -m log2(e) rounded to FP32, |r| <= 2^6 where |m| < 2^30.  The linear term of 2^r
// alone, which is enough near 0, is 1e-5 off at logits of 1e5 and has nothing to do with it at 3e7.
__device__ __forceinline__ float offset_factor(float m, float neg) {
    const float r = fmaf(-m, kLog2e, -neg), n = rintf(r);  // exact
    const float f = 1.f + expm1f((r - n) * kLn2);
    return f * __int_as_float((127 + int(n)) << 23);
}

// make_scale of the temperature 1
__device__ __forceinline__ Scale natural(float m) { return {m, 1.44269502162933349609375f, 1.92596299e-8f}; }

__device__ __forceinline__ uint64_t heavy_weight(const Scale& sc, float z, const RowArgs& a, const uint64_t* table) {
    return log2_weight(sc, z) > a.least_log2 ? weight_of(sc, z, table, a.q_bits) : 0;
}

__device__ __forceinline__ void add_mass(uint64_t* at, uint64_t w) {
    atomicAdd(reinterpret_cast<unsigned long long*>(at), static_cast<unsigned long long>(w));
}

// Sorts list[0 .. n), n <= kCap, descending.  All threads; the serving warp only waits.
__device__ __noinline__ void sort_block(uint64_t* list, int n) {
    const int t = int(threadIdx.x), step0 = t < kThreads ? t : kCap;
    int size = 2;
    while (size < n) size *= 2;
    __syncthreads();
    for (int i = n + step0; i < size; i += kThreads) list[i] = 0;
    __syncthreads();
    for (int len = 2; len <= size; len *= 2)
        for (int step = len / 2; step > 0; step /= 2) {
            for (int i = step0; i < size / 2; i += kThreads) {
                const int lo = (i / step) * step * 2 + i % step, hi = lo + step;
                const uint64_t a = list[lo], b = list[hi];
                if ((a < b) == ((lo & len) == 0)) list[lo] = b, list[hi] = a;
            }
            __syncthreads();
        }
}

// A block with more elements at or above the bound than the list holds (equal logits, or a
// few groups that have them all): element by element, the best ``count`` so far are kept
// whenever the list fills.  Their weights all enter the mass.  The part is copied again, as what
// was collected is gone from shared memory.  Rare, and kept out of the common code.  False when
// the copy did not arrive.
template <typename T>
__device__ __noinline__ bool collect_many(const RowArgs& a, Shared& sh, Part<T>& part, float part_max, float bound) {
    constexpr int VE = Part<T>::VE;
    const Scale sc = natural(part_max);
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
            sort_block(sh.list, int(n));
            if (threadIdx.x == 0) sh.n_list = uint32_t(a.count);
            least = sh.list[a.count - 1];
            __syncthreads();
        }
    };
    const int single = part.single();
    take(part.single_value(single), single);
    const int chunks = part.chunks();
    for (int c = 0; c < chunks; ++c) {
        if (!part.next(c)) return false;
#pragma unroll 1
        for (int j = 0; j < kHold * VE; ++j) {
            const int i = threadIdx.x < kThreads ? part.place(int(threadIdx.x), j) : -1;
            take(i >= 0 ? one(part.element_at(i)) : -INFINITY, part.token(c, i));
        }
    }
    add_mass(&sh.mass, mass);
    __syncthreads();
    return true;
}

// A copy that did not arrive in time: it may still write to shared memory, so the block waits for
// it, with a longer limit, before it goes.
template <typename T>
__device__ __noinline__ void lost(const Part<T>& part, int* dev_status) {
    if (threadIdx.x == 0) {
        report(dev_status, VCE_DEVSTATUS_TIMEOUT);
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&part.sh->arrived, part.parity ^ 1) && globaltimer() - t0 < kDrainTimeoutNs) {}
    }
    __syncthreads();
}

// The bound: the ``n``-th largest of the groups' maxima, n <= 16 of 32 groups or n <= 64 of 128;
// ``*top`` becomes the largest.  One warp: a lane holds one, or four in
// descending order, and gives up its largest when it is the largest of all.
template <int PER>
__device__ __forceinline__ uint32_t find_bound(const uint32_t* group, int n, uint32_t* top) {
    const int lane = threadIdx.x & 31;
    uint32_t t0, t1 = 0, t2 = 0, t3 = 0, best = 0;
    if constexpr (PER == 1) {
        t0 = group[lane];
    } else {
        const uint4 w = reinterpret_cast<const uint4*>(group)[lane];
        const uint32_t a = max(w.x, w.y), b = min(w.x, w.y), c = max(w.z, w.w), d = min(w.z, w.w);
        const uint32_t e = min(a, c), f = max(b, d);
        t0 = max(a, c), t1 = max(e, f), t2 = min(e, f), t3 = min(b, d);
    }
    for (int i = 0; i < n; ++i) {
        best = __reduce_max_sync(0xffffffffu, t0);
        if (i == 0) *top = best;
        const uint32_t who = __ballot_sync(0xffffffffu, t0 == best);
        if (lane == __ffs(int(who)) - 1) t0 = t1, t1 = t2, t2 = t3, t3 = 0;
    }
    return best;
}

template <typename T>
__global__ void __launch_bounds__(kThreads + 32, kBlocks) ce_beam_rows(const __grid_constant__ RowArgs a) {
    __shared__ Shared sh;
    extern __shared__ __align__(128) uint4 data[];
    constexpr int VE = 16 / sizeof(T);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool serves = warp == kWarps;
    const int64_t row = blockIdx.x, id = row * a.parts + blockIdx.y;
    const int rank = int(blockIdx.y);
    cudaTriggerProgrammaticLaunchCompletion();
    const float score = a.score[row];
    if (score == -INFINITY || (a.ended && a.ended[row])) return;  // nothing to read: the merge knows

    Part<T> part;
    part.row = static_cast<const T*>(a.logits) + row * a.stride;
    part.data = data, part.sh = &sh;
    part.off = int(reinterpret_cast<uintptr_t>(part.row) / sizeof(T) % VE);
    part.vocab = a.vocab;
    const int end = max(a.vocab / VE - 1, 1);
    part.g0 = min(end, 1 + rank * a.per), part.g1 = min(end, 1 + (rank + 1) * a.per);
    part.first = rank == 0, part.last = rank == a.parts - 1;
    part.dev_status = a.dev_status;
    part.parity = 0;
    if (tid == kThreads) {
        mbar_init(&sh.arrived, 1);
        fence_mbar_init();
        part.start(0);
        sh.n_list = 0, sh.n_hot = 0, sh.mass = 0, sh.abort = 0;
    }
    if (tid < kSteps) sh.table[tid] = kExp2Table[tid];
    const int single = part.single();
    float z1 = part.single_value(single);
    __syncthreads();

    // ---- the largest logit, and the largest of every thread's elements ----
    // A NaN stays the largest, and so it does as order_bits.
    const int chunks = part.chunks();
    float m = z1;
    bool ok = part.wait(0);
#pragma unroll 1
    for (int c = 0;;) {  // the last chunk stays
        if (serves) {
        } else if constexpr (sizeof(T) == 2) {
            uint32_t w = 0xff80ff80u;
            part.each([&](uint4 v) { w = max2_nan(w, max2_nan(max2_nan(v.x, v.y), max2_nan(v.z, v.w))); });
            m = max_nan(m, max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
        } else {
            part.each([&](uint4 v) {
                m = max_nan(max_nan(m, max_nan(__uint_as_float(v.x), __uint_as_float(v.y))),
                            max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
            });
        }
        if (++c == chunks || !ok) break;
        ok = part.next(c);
    }
    if (!serves) {
        uint32_t g = m == m ? order_bits(m + 0.f) : 0xffffffffu;
#pragma unroll
        for (int o = 1; o < kThreads / 128; o *= 2) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (a.count <= 16) {
#pragma unroll
            for (int o = kThreads / 128; o < kThreads / 32; o *= 2) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
            if (tid % (kThreads / 32) == 0) sh.group[tid / (kThreads / 32)] = g;
        } else if (tid % (kThreads / 128) == 0) {
            sh.group[tid / (kThreads / 128)] = g;
        }
    }
    __syncthreads();
    if (serves) {
        uint32_t top;
        const uint32_t best = a.count <= 16 ? find_bound<1>(sh.group, a.count, &top) : find_bound<4>(sh.group, a.count, &top);
        if (lane == 0) sh.bound = from_order_bits(best), sh.top = from_order_bits(top);
    }
    __syncthreads();
    const float bound = sh.bound, part_max = sh.top;
    PartHead* const head = a.heads + id;
    if (!ok || !(part_max < INFINITY) || part_max == -INFINITY) {  // nothing allowed here, or no distribution
        if (tid == 0) *head = {-INFINITY, ok && part_max == -INFINITY ? 0 : -1, 0};
        if (!ok) lost(part, a.dev_status);
        return;
    }

    // ---- the keys of the elements at or above the bound ----
    // Few threads have any: all threads look through what those few hold, and take out what they find.
    const Scale sc = natural(part_max);
    auto collect = [&](float z, int i) {
        const uint32_t at = atomicAdd(&sh.n_list, 1u);
        if (at < uint32_t(kCap)) sh.list[at] = key_of(z, i);
    };
    if (m >= bound && !serves) {
        if (z1 >= bound && z1 > -INFINITY) {
            collect(z1, single);
            z1 = -INFINITY;
        }
        sh.hot[atomicAdd(&sh.n_hot, 1u)] = uint16_t(tid);
    }
    __syncthreads();
    const int found = int(sh.n_hot) * (kHold * VE);
    // ---- the sum of the weights below it ----
    // (so far from 0 FP32 numbers are 64 apart, which no weight survives: only logits equal to the largest count)
    const bool near = fabsf(part_max) < 0x1p30f;
    const float neg = near ? -part_max * kLog2e : -INFINITY;
    const float2 log2e = make_float2(kLog2e, kLog2e), shift = make_float2(neg, neg);
    uint64_t* const keys = a.keys + id * a.count;
    float2 sum[2] = {};
    uint64_t mass = 0;  // of the serving warp
    float factor = 1.f;
    if (serves && near) factor = offset_factor(part_max, neg);
#pragma unroll 1
    for (int c = chunks - 1;;) {
        for (int j = tid; j < found; j += kThreads + 32) {
            const int i = part.place(sh.hot[j / (kHold * VE)], j % (kHold * VE));
            if (i < 0) continue;
            T* const at = part.element_at(i);
            const float z = one(at);
            if (z >= bound && z > -INFINITY) {
                collect(z, part.token(c, i));
                *at = T(-INFINITY);
            }
        }
        __syncthreads();
        if (!serves) {
            part.each([&](uint4 v) {
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    const float2 x = __ffma2_rn(make_float2(element<T>(v, e), element<T>(v, e + 1)), log2e, shift);
                    sum[e / 2 & 1] = __fadd2_rn(sum[e / 2 & 1], make_float2(ex2f(x.x), ex2f(x.y)));
                }
            });
        } else if (c == 0 && sh.n_list <= uint32_t(kFew)) {  // meanwhile the keys are sorted: each counts those before it
            const uint32_t n = sh.n_list;
            for (uint32_t i = lane; i < n; i += 32) {
                const uint64_t key = sh.list[i];
                mass += heavy_weight(sc, key_logit(key), a, sh.table);
                int before = 0;
#pragma unroll 8
                for (uint32_t j = 0; j < n; ++j) before += sh.list[j] > key;
                if (before < a.count) keys[before] = key;
            }
        }
        if (--c < 0 || !ok) break;
        ok = part.next(c);
    }
    if (!serves) {
        const float2 s = __fadd2_rn(sum[0], sum[1]);
        float total = s.x + s.y + ex2f(fmaf(z1, kLog2e, neg));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) sh.warp_sum[warp] = total;
    }
    __syncthreads();
    uint32_t n = sh.n_list;
    if (ok && n > uint32_t(kFew)) {
        if (n > uint32_t(kCap)) {
            ok = collect_many(a, sh, part, part_max, bound);
            n = sh.n_list;
        } else {
            for (uint32_t i = tid; i < n; i += kThreads + 32)
                add_mass(&sh.mass, heavy_weight(sc, key_logit(sh.list[i]), a, sh.table));
        }
        sort_block(sh.list, int(n));
        for (int i = tid; i < min(int(n), a.count); i += kThreads + 32) keys[i] = sh.list[i];
    }
    if (!ok) {
        if (tid == 0) *head = {-INFINITY, -1, 0};
        lost(part, a.dev_status);
        return;
    }
    if (!serves) return;
    // the light sums, as whole numbers
    if (lane < kWarps) mass += __float2ull_rn(sh.warp_sum[lane] * factor * __int_as_float((127 + a.q_bits) << 23));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    if (lane == 0) *head = {part_max, min(int(n), a.count), sh.mass + mass};
}

// ---------------------------------------------------------------------------
// the merge
// ---------------------------------------------------------------------------

struct MergeArgs {
    int64_t batch;
    int beams, count, parts, end, keep, q_bits;
    double penalty;
    float least_log2;
    const PartHead* heads;
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

// The lanes with the largest value; none when all are 0.
__device__ __forceinline__ uint32_t best_lanes(uint64_t value) {
    const uint32_t high = __reduce_max_sync(0xffffffffu, uint32_t(value >> 32));
    const uint32_t low = __reduce_max_sync(0xffffffffu, uint32_t(value >> 32) == high ? uint32_t(value) : 0u);
    return (high | low) == 0 ? 0u : __ballot_sync(0xffffffffu, value == (uint64_t(high) << 32 | low));
}

struct Row {  // of a request
    uint64_t mass;
    double log_s, norm;
    float m, score;
    int length;
    uint8_t ended, read, bad;
};

__device__ __forceinline__ double total_of(const Row& row, uint64_t key) {
    return double(row.score) + ((double(key_logit(key)) - double(row.m)) - row.log_s);
}

// One block per request.  Lists of candidates are merged by a warp, a lane to a list: the parts' lists
// of all beams at once where they are at most 32, otherwise first those of each beam.  FP64 is slow
// here, so what takes it is done for all rows, then for all candidates side by side.
__global__ void __launch_bounds__(kMergeThreads) ce_beam_merge(const __grid_constant__ MergeArgs a) {
    extern __shared__ uint64_t keys[];  // [beams][parts][count]; behind them the values of the lists to merge
    __shared__ uint64_t table[kSteps];
    __shared__ Row rows[kMaxBeams];
    __shared__ int part_n[kMaxBeams * kMaxParts], list_n[kMaxBeams];
    __shared__ int chosen_key[kMaxCount], chosen_parent[kMaxCount], place[kMaxCount];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t request = blockIdx.x;
    const int lists = a.beams * a.parts, all = lists * a.count;
    const bool at_once = lists <= 32;
    const int joined = at_once ? lists : a.beams;  // lists to merge, and
    uint64_t* const values = keys + all;
    int* const merged = reinterpret_cast<int*>(values + a.beams * a.count);  // where a beam's are merged first, their places
    // the search's state, which the kernel before does not write
    if (tid < kSteps) table[tid] = kExp2Table[tid];
    if (tid < a.beams) {
        const int64_t r = request * a.beams + tid;
        Row row{};
        row.score = a.score[r];
        row.ended = a.ended && a.ended[r];
        row.length = a.length ? a.length[r] : 0;
        row.read = row.score != -INFINITY && !row.ended;
        row.bad = row.score != -INFINITY && !(row.score < INFINITY && row.score > -INFINITY);
        row.norm = 1.0;
        if (a.penalty != 0.0) row.norm = pow(fmax(double(row.length) + !row.ended, 1.0), a.penalty);
        rows[tid] = row;
    }
    __syncthreads();
    cudaGridDependencySynchronize();
    auto head_of = [&](int r) {
        if (r < a.beams && lane < a.parts && rows[r].read) return a.heads[(request * a.beams + r) * a.parts + lane];
        return PartHead{-INFINITY, 0, 0};
    };
    PartHead coming = warp < kRowWarps ? head_of(warp) : PartHead{-INFINITY, 0, 0};  // on its way with the keys
    for (int i = tid; i < all; i += kMergeThreads)
        keys[i] = a.keys[request * all + i];  // (those past a list's number, and an ended beam's, are not looked at)
    for (int r = warp; r < a.beams && warp < kRowWarps; r += kRowWarps) {  // a row's parts
        const bool read = rows[r].read;
        const PartHead head = coming;
        coming = head_of(r + kRowWarps);
        const bool broken = __any_sync(0xffffffffu, head.n < 0);
        float m = head.m;
#pragma unroll
        for (int o = kMaxParts / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = __shfl_sync(0xffffffffu, m, 0);
        const bool bad = rows[r].bad || (read && (broken || m == -INFINITY));
        uint64_t mass = 0;
        if (read && !bad && head.m > -INFINITY) {
            const Scale sc = natural(m);
            if (log2_weight(sc, head.m) > a.least_log2) {
                const uint64_t w = weight_of(sc, head.m, table, a.q_bits);  // at most 2^Q
                mass = __umul64hi(head.mass, w) << (64 - a.q_bits) | head.mass * w >> a.q_bits;
            }
        }
#pragma unroll
        for (int o = kMaxParts / 2; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
        if (lane < a.parts) part_n[r * a.parts + lane] = bad ? 0 : rows[r].ended ? lane == 0 && rows[r].score > -INFINITY : head.n;
        if (lane == 0) {
            rows[r].mass = read && !bad ? mass : uint64_t(1) << a.q_bits;
            rows[r].m = m;
            if (bad) report(a.dev_status, VCE_DEVSTATUS_BAD_ROW);
        }
    }
    __syncthreads();
    if (warp == kRowWarps) {
        if (lane < a.beams) rows[lane].log_s = log(double(rows[lane].mass)) - a.q_bits * 0.69314718055994530942;
    } else if (!at_once) {
        for (int r = warp; r < a.beams; r += kRowWarps) {
            int at = (r * a.parts + lane) * a.count, n = 0;
            const int end = lane < a.parts ? at + part_n[r * a.parts + lane] : 0;
            uint64_t key = at < end ? keys[at] : 0;
            if (rows[r].ended) {
                n = part_n[r * a.parts];
                if (lane == 0) merged[r * a.count] = at;
            } else {
                for (; n < a.count; ++n) {
                    const uint32_t best = best_lanes(key);
                    if (best == 0) break;
                    if (best >> lane & 1) {  // (no two keys are equal)
                        merged[r * a.count + n] = at;
                        ++at;
                        key = at < end ? keys[at] : 0;
                    }
                }
            }
            if (lane == 0) list_n[r] = n;
        }
    }
    __syncthreads();
    for (int i = tid; i < joined * a.count; i += kMergeThreads) {
        const int list = i / a.count, n = at_once ? part_n[list] : list_n[list];
        if (i - list * a.count >= n) continue;
        const Row& row = rows[at_once ? list / a.parts : list];
        const double c = row.ended ? double(row.score) : total_of(row, keys[at_once ? i : merged[i]]);
        values[i] = order_bits(a.penalty != 0.0 ? c / row.norm : c);
    }
    __syncthreads();
    if (warp > 0) return;

    // ---- a lane's list, and its best candidate that has not been taken ----
    const int per = at_once ? a.parts : 1;
    int at = lane * a.count;
    const int end = lane < joined ? at + (at_once ? part_n[lane] : list_n[lane]) : 0;
    uint64_t value = at < end ? values[at] : 0;  // 0: none
    uint32_t taken = 0;
    uint64_t deferred = 0;  // chosen ones without a place of their own
    for (int i = 0; i < a.count; ++i) {
        uint32_t equal = best_lanes(value);
        int best = __ffs(int(equal)) - 1;
        if (equal & (equal - 1)) {  // the lowest beam, and in it the larger logit, which FP64 did not tell apart
            const bool mine = (equal >> lane & 1) && lane / per == best / per;
            uint64_t key = mine;  // (an ended beam has no key, and one list; no key is 0)
            if (mine && at_once && !rows[lane / per].ended) key = keys[at];
            best = __ffs(int(best_lanes(key))) - 1;
        }
        if (best < 0) {
            if (lane == 0) chosen_parent[i] = -1;
            deferred |= uint64_t(1) << i;
        } else {
            const int parent = best / per;
            if (taken >> parent & 1) deferred |= uint64_t(1) << i;
            taken |= 1u << parent;
            if (lane == best) {
                chosen_key[i] = at_once ? at : merged[at], chosen_parent[i] = parent, place[i] = parent;
                ++at;
                value = at < end ? values[at] : 0;
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
    for (int i = lane; i < a.count; i += 32) {
        const bool valid = chosen_parent[i] >= 0;
        const int to = a.keep ? place[i] : i, parent = valid ? chosen_parent[i] : to % a.beams;
        const Row& row = rows[parent];
        const int64_t out = request * a.count + to;
        int token = -1;
        double c = -INFINITY;
        if (valid && row.ended) token = a.end, c = double(row.score);
        else if (valid) token = key_index(keys[chosen_key[i]]), c = total_of(row, keys[chosen_key[i]]);
        a.token[out] = token;
        a.parent[out] = parent;
        a.out_score[out] = float(c);
        if (a.out_ended) a.out_ended[out] = valid && (row.ended || token == a.end);
        if (a.out_length) a.out_length[out] = row.length + (valid && !row.ended && row.length < INT_MAX);
    }
}

size_t merge_bytes(int beams, int count, int parts) {
    return size_t(beams) * count * (beams * parts <= 32 ? parts * 16 : parts * 8 + 12);
}

// A row in as many parts as let each fit a block's shared memory, and as fill the SMs where rows are
// few (each with some vectors for every thread).
int parts_of(int64_t rows, int beams, int count, int64_t vocab, int dtype, int num_sms) {
    const int64_t vectors = vocab / (dtype == VCE_BF16 ? 8 : 4), whole = (vectors + kHold * kThreads - 1) / (kHold * kThreads);
    const int64_t fill = std::min<int64_t>(2 * num_sms / rows, vectors / (2 * kThreads));
    int parts = int(std::max<int64_t>(1, std::min<int64_t>(kMaxParts, std::max(whole, fill))));
    while (merge_bytes(beams, count, parts) > kMergeBytes) --parts;
    return parts;
}

}  // namespace

size_t ce_beam_ws_bytes(int64_t rows, int count) {
    return align256(size_t(rows) * kMaxParts * sizeof(PartHead)) + size_t(rows) * kMaxParts * size_t(count) * sizeof(uint64_t);
}

vce_status launch_ce_beam(const void* logits, int dtype, int64_t batch, int beams, int64_t vocab, int64_t stride,
                          const float* score, const uint8_t* ended, const int* length, int64_t end, double penalty,
                          int count, int keep, int64_t* token, int64_t* parent, float* out_score,
                          uint8_t* out_ended, int* out_length, void* ws, int* dev_status, cudaStream_t s,
                          const DeviceInfo& dev) {
    const int64_t rows = batch * beams;
    if (rows == 0) return VCE_OK;
    int bits = 0;
    while ((int64_t(1) << bits) < vocab) ++bits;
    const int q_bits = 63 - bits < 44 ? 63 - bits : 44, parts = parts_of(rows, beams, count, vocab, dtype, dev.num_sms);
    const int64_t groups = std::max<int64_t>(vocab / (dtype == VCE_BF16 ? 8 : 4) - 2, 0);
    const RowArgs a{logits, stride, int(vocab), score, ended, count, parts, int((groups + parts - 1) / parts), q_bits, -float(q_bits + 1) + 0x1p-10f,
                    static_cast<PartHead*>(ws),
                    reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + align256(size_t(rows) * kMaxParts * sizeof(PartHead))),
                    dev_status};
    static std::mutex mu;
    static bool ready[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev.ordinal]) {
            const auto most = cudaFuncAttributeMaxDynamicSharedMemorySize;
            if (cudaFuncSetAttribute(ce_beam_rows<__nv_bfloat16>, most, kBytes) != cudaSuccess ||
                cudaFuncSetAttribute(ce_beam_rows<float>, most, kBytes) != cudaSuccess ||
                cudaFuncSetAttribute(ce_beam_merge, most, kMergeBytes) != cudaSuccess)
                return VCE_ERR_CUDA;
            ready[dev.ordinal] = true;
        }
    }
    count_launch();
    const dim3 grid{unsigned(rows), unsigned(parts)};
    if (dtype == VCE_BF16) ce_beam_rows<__nv_bfloat16><<<grid, kThreads + 32, kBytes, s>>>(a);
    else ce_beam_rows<float><<<grid, kThreads + 32, kBytes, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return VCE_ERR_CUDA;

    const MergeArgs g{batch, beams, count, parts, int(end), keep, q_bits, penalty, a.least_log2, a.heads, a.keys, score,
                      ended, length, token, parent, out_score, out_ended, out_length, dev_status};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(batch));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = merge_bytes(beams, count, parts);
    cfg.stream = s;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, ce_beam_merge, g) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
