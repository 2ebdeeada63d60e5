// Sampling of one token per row of logits with temperature, top-k, top-p and min-p
// from a given uniform number.
//
// The tokens of a row are ordered by (logit descending, index ascending).  Every filter
// keeps a head of that order, so all of them together do too, and the token is the
// first of the head whose cumulated weight exceeds u times the head's.
//
// Weights are whole numbers.  The choice compares sums of up to 2^20 weights with a
// border that lies between two of them; FP32 sums would move it by whole tokens, and a
// result would depend on the order of additions.  Weight i is
//     2^(Q + n / 64) s / 2^36,  n / 64 + log2(s / 2^36) = (z_i - m) c,  c = log2(e) / T,
// with n and s whole and s within 2^-36 of its exact value (relative) (step_of below).  Q is at most
// 44 and leaves room for the sum of a row (2^63).  Integer sums come out the same in any order: the
// row is split over threads and blocks freely, and atomics change nothing.  They are rounded,
// though: a mass (below) as a whole, far down of s in steps of 2^7, a sorted token's weight by
// itself.  Where both meet, a head's mass is kept from passing that of its last n.
//
// A row never gets sorted as a whole:
//   heads  (top-k up to kMaxHeads, or min-p without top-p): a bound is found below
//          which nothing survives - the k-th largest of the maxima of disjoint groups
//          of elements, or min-p's own - and what lies above it, a little more than the
//          head, is collected and sorted in shared memory.
//   masses (otherwise): for every n the sum of its elements' s is collected by 32-bit
//          atomics; n is ordered by construction and the scaling by 2^(n / 64) happens
//          once per n.  A border is located among the
//          prefix sums of the masses, and only the elements of that one n are collected
//          and sorted.  Too many of them are divided again by the bits of (logit, index).
// The logits are read once from HBM; the later passes find them in L2.
//
// What bounds it is not the memory but, for few rows, the chain of short serial steps
// (1 x 128256 BF16, top-k and top-p: 18 us), and for many the instructions and
// shared-memory atomics of the pass that sums masses (1024 x 50257 FP32, no filter: 195 us,
// 31 us at the copy rate; with sums in 64-bit atomics 377 us).
//
// A row is shared by a cluster of blocks (one when there are rows enough).  Block 0 joins
// the others' results, which it reads from their shared memory, and decides; the others
// read its decision.

#include "head_internal.cuh"
#include "sm100_ptx.cuh"

#include <math.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 64;            // values of n per octave
constexpr int kBins = 46 * kSteps;    // 46 octaves of n, from 0 down
constexpr int kFracBits = 36;         // of s
constexpr int kBiasBits = 29;         // s - 2^36 is above -2^29 and below 2^29
// Sums of s are kept in 32-bit words of 15 bits of every s, which 2^17 elements cannot
// overflow.  The 8 octaves below the largest logit get s - 2^36 + 2^29 in two words and
// a count; further down 30 bits of s itself are enough (2^-29 of a weight that is at most
// 2^-8), two words and no count.
constexpr int kHalfBits = 15;
constexpr int kMaxPart = 1 << 17;     // elements per block, at most
constexpr int kFineBins = 8 * kSteps;
constexpr int kCoarseBits = 7;        // of s, rounded away further down
constexpr uint32_t kCoarseOffset = (1u << (kFracBits - kCoarseBits)) - (1u << (kBiasBits - kCoarseBits));  // 2^36 - 2^29 there
constexpr int kCap = 2048;          // collected elements; also sub-bins of a divided bin
constexpr int kCapBits = 11;
constexpr int kMaxHeads = 256;      // top-k of the collecting path
constexpr int kIndexBits = 20;      // vocabulary of at most 2^20
constexpr int kMaxCluster = 8;
constexpr int kEdgeBins = 5;       // around min-p's border: weights there are compared one by one

__device__ const uint64_t kExp2Table[kSteps] = {
#include "exp2_table.inc"
};

struct SampleArgs {
    const void* logits;
    int64_t n, stride;
    int vocab;
    const float *uniform, *temperature, *top_p, *min_p;
    const int* top_k;
    int64_t* token;
    float* logprob;
    int cluster;
    int q_bits;  // Q
    float least_log2;  // weights above it round to one unit 2^-Q at least, others count as 0
    int* dev_status;
};

// What block 0 tells the others.
struct Command {
    uint64_t lo, hi;  // range of (logit, index) keys
    int bin, flag;
};

// Which elements to collect: logits in [z_lo, z_hi] with a log2_weight above p_least, in
// ``cmd``'s range of keys and, unless its bin is negative, in its bin.
struct Wanted {
    float z_lo, z_hi, p_least;
    Command cmd;
};

struct Shared {
    uint64_t mass[kBins];  // words of low and then of high halves, then the sum of s, then (block 0) prefix sums of masses
    uint32_t count[kBins];  // for top-k and the last kept; the first kFineBins always
    uint64_t list[kCap];   // collected keys; masses of sub-bins
    uint64_t sums[kCap];   // inclusive prefix sums of the sorted list; counts of sub-bins
    uint64_t table[kSteps];
    uint64_t warp_sum[kWarps];
    float group[kThreads];
    float warp_max[kWarps];
    // written by every block into every block's memory, each into the slot of its rank, once
    float row_max[kMaxCluster], bound[kMaxCluster];
    Command cmd[2];  // by block 0; consecutive commands take turns: a late reader finds its own intact
    uint32_t part_n[kMaxCluster];  // block 0's: what the others have collected
    uint64_t min_key, max_key;
    uint64_t kept_minp[kEdgeBins];  // sums of the weights that min-p keeps, per bin, and
    uint32_t kept_n[kEdgeBins];     // how many they are
    float my_bound;
    uint32_t n_list, found, argmax;
    uint32_t n_kept, n_above;  // block 0's: tokens that top-k and top-p keep, and min-p
};

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t order_bits(float z) {  // monotone in z
    const uint32_t b = __float_as_uint(z);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// (logit, index) as one number: larger comes first.  -0 counts as 0.
__device__ __forceinline__ uint64_t key_of(float z, int i) {
    return uint64_t(order_bits(z + 0.f)) << kIndexBits | uint32_t((1 << kIndexBits) - 1 - i);
}
__device__ __forceinline__ float key_logit(uint64_t k) { return from_order_bits(uint32_t(k >> kIndexBits)); }
__device__ __forceinline__ int key_index(uint64_t k) { return (1 << kIndexBits) - 1 - int(k & ((1 << kIndexBits) - 1)); }

// A row's scale: m its largest logit, ch + cl = log2(e) / T as an unevaluated sum.
struct Scale {
    float m, ch, cl;
};

__device__ __forceinline__ Scale make_scale(float m, float t) {
    const float lh = 1.44269502162933349609375f, ll = 1.92596299e-8f;  // log2(e) = lh + ll
    t = fminf(fmaxf(t, 1e-30f), 1e30f);
    const float ch = lh / t;
    const float r = fmaf(-ch, t, lh) + ll;  // the division's remainder, exact
    return {m, ch, r / t};
}

// The leading term of (z - m) c, monotone in z.
__device__ __forceinline__ float log2_weight(const Scale& s, float z) { return __fmul_rn(z - s.m, s.ch); }

// The element's n (as the bin -n) and s of a log2_weight above least_log2.
//   (z - m) and its product with c are carried as sums of two floats (TwoSum, FMA), about
//   2^-47 relative.  The exponent is n / 64 + f with |f| <= 2^-7; 2^f - 1 from its series
//   to the fifth power, its linear term split into a multiple of 2^-29 and a rest.
//   round(64 p) is taken by adding 1.5 x 2^23.
__device__ __forceinline__ int bin_of(float p) { return 0x4b400000 - __float_as_int(fmaf(p, float(kSteps), 12582912.f)); }

struct Step {
    int bin;
    int g;  // s - 2^kFracBits
};
__device__ __forceinline__ Step step_of(const Scale& s, float z) {
    const float d = z - s.m;
    const float b = d - z;
    const float dl = (z - (d - b)) - (s.m + b);
    const float p = __fmul_rn(d, s.ch);
    float e = fmaf(d, s.ch, -p);
    e = fmaf(d, s.cl, e);
    e = fmaf(dl, s.ch, e);
    const float t = fmaf(p, float(kSteps), 12582912.f);
    const float f = fmaf(t - 12582912.f, -1.f / kSteps, p);
    const float lh = 0.693147182464599609375f, ll = -1.904654323148236e-9f;  // ln 2 = lh + ll
    const float a = f * lh;
    float r = fmaf(f, lh, -a);
    r = fmaf(f, ll, r);
    r = fmaf(e, lh, r);
    // ln2^k / k! for k = 2 .. 5
    const float c2 = 0.24022650695910072f, c3 = 0.05550410866482158f, c4 = 0.009618129107628477f,
                c5 = 0.0013333558146428443f;
    const float fe = f + e;
    r = fmaf(fe * fe, fmaf(fmaf(fmaf(c5, f, c4), f, c3), f, c2), r);
    const float big = 1.5f * 0x1p-6f;  // |a| < 2^-7: the sum stays in big's binade, whose last bit is 2^-29
    const float u = a + big;
    const int hi = __float_as_int(u) - __float_as_int(big);
    r += a - (u - big);
    const int lo = __float_as_int(fmaf(r, 0x1p36f, 12582912.f)) - 0x4b400000;
    return {0x4b400000 - __float_as_int(t), hi * 128 + lo};
}

// step_of for two logits at once, two lanes to an instruction, and with the signs turned:
// x = (m - z) c = P + E is not negative, F = P - bin / 64, and 2^-(F + E) - 1 is wanted.
// ``s`` is s + 2^29 - 2^36, not negative.
struct Step2 {
    float2 p;
    int bin[2];
    uint32_t s[2];
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ Step2 step_of2(const Scale& sc, float2 z) {
    const float2 minus = both(-1.f), m = both(sc.m);
    const float2 d = __fadd2_rn(z, both(-sc.m));
    const float2 b = __ffma2_rn(z, minus, d);
    const float2 dl = __ffma2_rn(__fadd2_rn(m, b), minus, __ffma2_rn(__ffma2_rn(b, minus, d), minus, z));
    const float2 nch = both(-sc.ch);
    const float2 p = __fmul2_rn(d, nch);
    float2 e = __ffma2_rn(d, nch, __fmul2_rn(d, both(sc.ch)));
    e = __ffma2_rn(d, both(-sc.cl), e);
    e = __ffma2_rn(dl, nch, e);
    const float2 t = __ffma2_rn(p, both(float(kSteps)), both(12582912.f));
    const float2 f = __ffma2_rn(__fadd2_rn(t, both(-12582912.f)), both(-1.f / kSteps), p);
    const float lh = 0.693147182464599609375f, ll = -1.904654323148236e-9f;
    const float2 a = __fmul2_rn(f, both(-lh));
    float2 r = __ffma2_rn(f, both(-lh), __fmul2_rn(f, both(lh)));
    r = __ffma2_rn(f, both(-ll), r);
    r = __ffma2_rn(e, both(-lh), r);
    const float2 fe = __fadd2_rn(f, e);
    float2 q = __ffma2_rn(f, both(-0.0013333558146428443f), both(0.009618129107628477f));
    q = __ffma2_rn(q, f, both(-0.05550410866482158f));
    q = __ffma2_rn(q, f, both(0.24022650695910072f));
    r = __ffma2_rn(__fmul2_rn(fe, fe), q, r);
    const float big = 1.5f * 0x1p-6f;
    const float2 u = __fadd2_rn(a, both(big));
    r = __fadd2_rn(r, __ffma2_rn(__fadd2_rn(u, both(-big)), minus, a));
    const float2 lo = __ffma2_rn(r, both(0x1p36f), both(12582912.f));
    const uint32_t off = (1u << kBiasBits) - 0x4b400000u - uint32_t(__float_as_int(big)) * 128u;
    return {p,
            {__float_as_int(t.x) - 0x4b400000, __float_as_int(t.y) - 0x4b400000},
            {uint32_t(__float_as_int(u.x)) * 128u + uint32_t(__float_as_int(lo.x)) + off,
             uint32_t(__float_as_int(u.y)) * 128u + uint32_t(__float_as_int(lo.y)) + off}};
}

// round(2^Q 2^(-bin / 64) sum / 2^36) for a sum of s below 2^57
__device__ __forceinline__ uint64_t scale_up(uint64_t sum, int bin, const uint64_t* table, int q_bits) {
    const int n = -bin;
    const uint64_t t = table[n & (kSteps - 1)];                       // 63 fractional bits
    const int shift = 63 + kFracBits - q_bits - (n >> 6);             // 55 .. 102
    const uint64_t hi = __umul64hi(sum, t), lo = sum * t;
    uint64_t q, rest;  // the value rounded down (2^63 for a row of full weights), and the bits below it from the top down
    if (shift < 64) {
        q = hi << (64 - shift) | lo >> shift;
        rest = lo << (64 - shift);
    } else {
        q = hi >> (shift - 64);
        rest = shift == 64 ? lo : hi << (128 - shift);
    }
    return q + (rest >> 63);
}

__device__ __forceinline__ uint64_t weight_of(const Scale& s, float z, const uint64_t* table, int q_bits) {
    const Step st = step_of(s, z);
    return scale_up((uint64_t(1) << kFracBits) + int64_t(st.g), st.bin, table, q_bits);
}

// floor(x y) for a float 0 <= x < 1 and y <= 2^63; ``*exact`` tells whether nothing was cut off
__device__ __forceinline__ uint64_t floor_product(float x, uint64_t y, bool* exact) {
    const uint32_t b = __float_as_uint(x);
    const int e = int(b >> 23) & 255;
    const uint64_t man = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int shift = 150 - (e ? e : 1);  // x = man 2^-shift, shift >= 24
    const uint64_t hi = __umul64hi(man, y), lo = man * y;  // hi < 2^23
    uint64_t q, cut;
    if (shift < 64) {
        q = hi << (64 - shift) | lo >> shift;
        cut = lo << (64 - shift);
    } else if (shift < 128) {
        q = shift == 64 ? hi : hi >> (shift - 64);
        cut = lo | (shift == 64 ? 0 : hi << (128 - shift));
    } else {
        q = 0;
        cut = hi | lo;
    }
    *exact = cut == 0;
    return q;
}

// This block's part of a row.  Vectors are 16 bytes at 16-byte aligned addresses; vector
// q holds elements q VE - off ....  The vectors that lie in the row as a whole are divided
// among the blocks, [q0, q1) to this one; the elements before and behind them are the last
// block's, which has fewest vectors: no block has more than kMaxPart elements.
template <typename T>
struct Part {
    const T* row;
    int off, vocab;
    int q0, q1;
    bool last;
};

template <typename T>
__device__ __forceinline__ float element(uint4 v, int e);
template <>
__device__ __forceinline__ float element<float>(uint4 v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
}
template <>
__device__ __forceinline__ float element<__nv_bfloat16>(uint4 v, int e) {
    const uint32_t w = (e >> 1) == 0 ? v.x : (e >> 1) == 1 ? v.y : (e >> 1) == 2 ? v.z : v.w;
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// fn(logit, logit, index) for every two neighbouring elements of the block's part (index is
// the first one's).  The vectors come first, then single elements, each with -inf beside it.  Short bodies take U vectors
// at a time, all of them loaded first; long ones (kAhead > 0) one, with the next kAhead on
// their way: their code, laid out several times, cost more in instruction fetches than
// the loads in flight gained.
template <int U, int kAhead = 0, typename T, typename F>
__device__ __forceinline__ void for_pairs(const Part<T>& p, int* dev_status, F fn) {
    constexpr int VE = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int end = p.q1;
    int q = p.q0 + tid;
    const T* at = p.row + (q * VE - p.off);
    auto fetch = [&](int k) {  // vector q + k kThreads
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q + k * kThreads < end && VCE_BOUNDS(aligned16(at), dev_status))
            v = __ldg(reinterpret_cast<const uint4*>(at + k * kThreads * VE));
        return v;
    };
    if constexpr (kAhead > 0) {  // long bodies, one vector at a time: the next ones are on their way
        uint4 ring[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) ring[k] = fetch(k);
#pragma unroll 1
        for (; q < end; q += kThreads, at += kThreads * VE) {
            const uint4 v = ring[0];
#pragma unroll
            for (int k = 0; k + 1 < kAhead; ++k) ring[k] = ring[k + 1];
            ring[kAhead - 1] = fetch(kAhead);
            const int i = q * VE - p.off;
#pragma unroll
            for (int e = 0; e < VE; e += 2) fn(element<T>(v, e), element<T>(v, e + 1), i + e);
        }
    } else {
        for (; q < end; q += U * kThreads, at += U * kThreads * VE) {
            uint4 v[U];
#pragma unroll
            for (int k = 0; k < U; ++k) v[k] = fetch(k);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (q + k * kThreads >= end) break;
                const int i = (q + k * kThreads) * VE - p.off;
#pragma unroll
                for (int e = 0; e < VE; e += 2) fn(element<T>(v[k], e), element<T>(v[k], e + 1), i + e);
            }
        }
    }
    // the first vector's elements, then those behind the whole vectors
    if (!p.last) return;
    const int whole = (p.off + p.vocab) / VE, first = p.off > 0 ? min(VE - p.off, p.vocab) : 0;
    const int tail0 = max(whole * VE - p.off, first);
    if (tid < first + max(p.vocab - tail0, 0)) {
        const int i = tid < first ? tid : tail0 + tid - first;
        fn(one(p.row + i), -INFINITY, i);
    }
}

// fn(logit, index) for every element; also for a -inf with the index after a single one's
template <int U, int kAhead = 0, typename T, typename F>
__device__ __forceinline__ void for_each(const Part<T>& p, int* dev_status, F fn) {
    for_pairs<U, kAhead>(p, dev_status, [&](float z0, float z1, int i) {
        fn(z0, i);
        fn(z1, i + 1);
    });
}

// the address of ``p`` (in shared memory) in block ``rank`` of the cluster
template <typename T>
__device__ __forceinline__ T remote(const T* p, int rank) {
    const uint32_t a = mapa_shared(smem_u32(p), uint32_t(rank));
    if constexpr (sizeof(T) == 8) {
        uint64_t v;
        asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
        return *reinterpret_cast<T*>(&v);
    } else {
        uint32_t v;
        asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
        return *reinterpret_cast<T*>(&v);
    }
}

__device__ __forceinline__ void put(uint64_t* p, int rank, uint64_t v) {
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), uint32_t(rank))), "l"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t* p, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), uint32_t(rank))), "r"(v) : "memory");
}

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void row_barrier(int cluster) {
    if (cluster == 1) __syncthreads();
    else cluster_sync();
}

// a[i] = the sum of load(0) ... load(i), i < n <= PER x kThreads; load(i) may read a[i].
// Every thread calls; each takes PER neighbours.
template <int PER, typename T, typename F>
__device__ __forceinline__ void prefix_sums(T* a, int n, uint64_t* warp_sum, F load) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = int(threadIdx.x) * PER;
    uint64_t v[PER], s = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        s += i0 + k < n ? uint64_t(load(i0 + k)) : 0;
        v[k] = s;
    }
    uint64_t t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += x;
    }
    if (lane == 31) warp_sum[warp] = t;
    __syncthreads();
    uint64_t before = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    before = __shfl_sync(0xffffffffu, before, 0) + t - s;  // lanes 0 .. 15 hold the sum of the warps'
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (i0 + k < n) a[i0 + k] = T(before + v[k]);
    __syncthreads();
}

// The first i < n with s[i] >= target in an ascending s (n when there is none); every
// thread finds it by itself.
template <typename V>
__device__ __forceinline__ int first_at_least(const V* s, int n, V target) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s[mid] >= target) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Sorts list[0 .. n), n <= kCap, descending (all keys differ); ``tmp`` is scratch.
__device__ __forceinline__ void sort_list(uint64_t* list, int n, uint64_t* tmp) {
    const int t = threadIdx.x;
    if (n <= kThreads / 2) {  // each key counts those before it, two threads to a key
        const int i = t >> 1, half = (n + 1) >> 1;
        const uint64_t k = i < n ? list[i] : 0;
        int r = 0;
        const int end = t & 1 ? n : half;
#pragma unroll 4
        for (int j = t & 1 ? half : 0; j < end; ++j) r += list[j] > k;
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        if (i < n && !(t & 1)) tmp[r] = k;
        __syncthreads();
        if (t < n) list[t] = tmp[t];
        __syncthreads();
        return;
    }
    int size = kThreads;
    while (size < n) size *= 2;
    for (int i = n + t; i < size; i += kThreads) list[i] = 0;  // after every key
    __syncthreads();
    if (size == kThreads) {  // one key per thread: partners within a warp need no barrier
        uint64_t key = list[t];
#pragma unroll 1
        for (int len = 2; len <= size; len *= 2)
#pragma unroll 1
            for (int step = len / 2; step > 0; step /= 2) {
                uint64_t other;
                if (step >= 32) {
                    __syncthreads();
                    list[t] = key;
                    __syncthreads();
                    other = list[t ^ step];
                } else {
                    other = __shfl_xor_sync(0xffffffffu, key, step);
                }
                const bool larger = ((t & len) == 0) == ((t & step) == 0);  // this place keeps the larger
                key = (other > key) == larger ? other : key;
            }
        __syncthreads();
        list[t] = key;
        __syncthreads();
        return;
    }
#pragma unroll 1
    for (int len = 2; len <= size; len *= 2)
#pragma unroll 1
        for (int step = len / 2; step > 0; step /= 2) {
            for (int i = t; i < size / 2; i += kThreads) {
                const int lo = (i / step) * step * 2 + i % step, hi = lo + step;
                const bool desc = (lo & len) == 0;
                const uint64_t a = list[lo], b = list[hi];
                if ((a < b) == desc) list[lo] = b, list[hi] = a;
            }
            __syncthreads();
        }
}

template <typename T>
struct Sampler {
    const SampleArgs& a;
    Shared& sh;
    Part<T> part;
    int rank;
    Scale sc;
    uint32_t turn;  // commands so far

    __device__ __forceinline__ bool lead() const { return rank == 0; }
    __device__ __forceinline__ void barrier() const { row_barrier(a.cluster); }

    // Block 0's command (the same in all its threads), in every block: it is put into their
    // shared memory before a barrier.  A slot is written again two commands later, behind
    // a barrier that its readers have passed.
    __device__ __forceinline__ Command tell(const Command& c) {
        Command* slot = &sh.cmd[turn & 1];
        ++turn;
        if (lead() && int(threadIdx.x) < a.cluster) {
            if (a.cluster == 1) {
                *slot = c;
            } else {
                put(&slot->lo, threadIdx.x, c.lo);
                put(&slot->hi, threadIdx.x, c.hi);
                put(reinterpret_cast<uint32_t*>(&slot->bin), threadIdx.x, uint32_t(c.bin));
                put(reinterpret_cast<uint32_t*>(&slot->flag), threadIdx.x, uint32_t(c.flag));
            }
        }
        barrier();
        return *slot;
    }

    __device__ __forceinline__ void take(const Wanted& w, float z, int i) {
        const float p = log2_weight(sc, z);
        const uint64_t k = key_of(z, i);
        if (p > w.p_least && (w.cmd.bin < 0 || bin_of(p) == w.cmd.bin) && k >= w.cmd.lo && k <= w.cmd.hi) {
            const uint32_t at = atomicAdd(&sh.n_list, 1u);
            if (at < kCap) sh.list[at] = k;
        }
    }

    // Collects the keys of the elements that are wanted; behind the barrier block 0 has
    // every block's number of them.
    __device__ __forceinline__ void collect(const Wanted& w) {
        if (threadIdx.x == 0) sh.n_list = 0;
        __syncthreads();
        const float z_lo = w.z_lo, z_hi = w.z_hi;
        for_each<1, 2>(part, a.dev_status, [&](float z, int i) {
            if (z >= z_lo && z <= z_hi) take(w, z, i);
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            if (lead()) sh.part_n[0] = sh.n_list;
            else put(&sh.part_n[rank], 0, sh.n_list);
        }
        barrier();
    }

    // Block 0: the others' lists behind its own.  False when they are too many.
    __device__ __forceinline__ bool join_lists(int& n) {
        uint32_t total = 0;
        for (int c = 0; c < a.cluster; ++c) total += sh.part_n[c];
        if (total > kCap) return false;
        n = int(total);
        if (a.cluster == 1) return true;
        for (uint32_t i = sh.part_n[0] + threadIdx.x; i < total; i += kThreads) {
            uint32_t c = 0, j = i;
            while (j >= sh.part_n[c]) j -= sh.part_n[c++];
            sh.list[i] = remote(&sh.list[j], int(c));
        }
        __syncthreads();
        return true;
    }

    __device__ __forceinline__ void add_mass(uint64_t* at, uint64_t w) {
        atomicAdd(reinterpret_cast<unsigned long long*>(at), static_cast<unsigned long long>(w));
    }

    // The elements of one bin.  The logits' bounds are generous; the bin itself decides.
    __device__ __forceinline__ Wanted in_bin(const Command& cmd) const {
        const float far = (float(cmd.bin) + 0.75f) / (kSteps * sc.ch), near = (float(cmd.bin) - 0.75f) / (kSteps * sc.ch);
        const float slack = fabsf(sc.m) * 0x1p-21f;
        return {sc.m - far - slack, sc.m - near + slack, a.least_log2, cmd};
    }

    // A range that holds more elements than a list: its keys divided into kCap ranges of
    // equal width, of which the one with the target is the new range.  ``base`` and
    // ``base_count`` become what lies before it.  Rare, and kept out of the common code.
    __device__ __noinline__ void divide(Command& cmd, bool by_count, uint64_t target, uint64_t& base,
                                        uint32_t& base_count) {
        const Wanted w = in_bin(cmd);
        auto mine = [&](float z, int i) {
            if (!(z >= w.z_lo && z <= w.z_hi)) return false;
            const float p = log2_weight(sc, z);
            const uint64_t k = key_of(z, i);
            return p > a.least_log2 && bin_of(p) == w.cmd.bin && k >= w.cmd.lo && k <= w.cmd.hi;
        };
        uint64_t kmin = ~0ull, kmax = 0;
        for_each<1>(part, a.dev_status, [&](float z, int i) {
            if (!mine(z, i)) return;
            const uint64_t k = key_of(z, i);
            kmin = k < kmin ? k : kmin;
            kmax = k > kmax ? k : kmax;
        });
        if (threadIdx.x == 0) sh.min_key = ~0ull, sh.max_key = 0;
        for (int i = threadIdx.x; i < kCap; i += kThreads) sh.list[i] = 0, sh.sums[i] = 0;
        __syncthreads();
        atomicMin(reinterpret_cast<unsigned long long*>(&sh.min_key), static_cast<unsigned long long>(kmin));
        atomicMax(reinterpret_cast<unsigned long long*>(&sh.max_key), static_cast<unsigned long long>(kmax));
        barrier();
        if (lead()) {
            cmd.lo = ~0ull, cmd.hi = 0;
            for (int c = 0; c < a.cluster; ++c) {
                const uint64_t x = remote(&sh.min_key, c), y = remote(&sh.max_key, c);
                cmd.lo = x < cmd.lo ? x : cmd.lo;
                cmd.hi = y > cmd.hi ? y : cmd.hi;
            }
        }
        cmd = tell(cmd);
        const uint64_t l = cmd.lo, h = cmd.hi;
        const int bits = 64 - __clzll(int64_t(h - l));
        const int shift = bits > kCapBits ? bits - kCapBits : 0;
        for_each<1>(part, a.dev_status, [&](float z, int i) {
            if (!mine(z, i)) return;
            const uint64_t b = (h - key_of(z, i)) >> shift;
            if (!VCE_BOUNDS(b < uint64_t(kCap), a.dev_status)) return;
            add_mass(&sh.list[b], weight_of(sc, z, sh.table, a.q_bits));
            add_mass(&sh.sums[b], 1);
        });
        barrier();
        if (lead()) {
            for (int i = threadIdx.x; i < kCap; i += kThreads)
                for (int c = 1; c < a.cluster; ++c) {
                    sh.list[i] += remote(&sh.list[i], c);
                    sh.sums[i] += remote(&sh.sums[i], c);
                }
            __syncthreads();
            prefix_sums<kCap / kThreads>(sh.list, kCap, sh.warp_sum, [&](int i) { return sh.list[i]; });
            prefix_sums<kCap / kThreads>(sh.sums, kCap, sh.warp_sum, [&](int i) { return sh.sums[i]; });
            // (the bin's mass, rounded once, can be more than the sum of its weights, rounded one
            // by one: a target between the two takes the last range that holds a key)
            const int b = min(by_count ? first_at_least(sh.sums, kCap, target - base_count)
                                       : first_at_least(sh.list, kCap, target > base ? target - base : 1),
                              int((h - l) >> shift));
            if (b > 0) base += sh.list[b - 1], base_count += uint32_t(sh.sums[b - 1]);
            const uint64_t width = (uint64_t(1) << shift) - 1;
            cmd.hi = h - (uint64_t(b) << shift);
            cmd.lo = cmd.hi - l > width ? cmd.hi - width : l;
        }
        cmd = tell(cmd);
    }

    __device__ __forceinline__ void write(int64_t row, int64_t token, float logprob) {
        a.token[row] = token;
        if (a.logprob) a.logprob[row] = logprob;
    }

    // Block 0, thread 0: the drawn token, of weight w, and the logarithm of its share of the mass.
    __device__ __forceinline__ void finish(int64_t row, uint64_t key, uint64_t w, uint64_t mass, float t) {
        write(row, key_index(key), 0.f);
        if (!a.logprob) return;
        const float z = key_logit(key);
        float lp;
        if (w > mass / 2) lp = log1pf(-__ull2float_rn(mass - w) / __ull2float_rn(mass));
        else lp = (z - sc.m) / fminf(fmaxf(t, 1e-30f), 1e30f) - logf(ldexpf(__ull2float_rn(mass), -a.q_bits));
        a.logprob[row] = lp;
    }
};

// What the collected lists are for, in this order: all survivors at once, or the border
// of top-k, that of top-p, the draw.
enum { kHeads, kTopK, kTopP, kDraw };

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) ce_sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const int tid = threadIdx.x;
    const int rank = a.cluster == 1 ? 0 : int(cluster_ctarank());
    const int64_t row = int64_t(blockIdx.x) / a.cluster;
    if (tid < kSteps) sh.table[tid] = kExp2Table[tid];

    constexpr int VE = 16 / sizeof(T);
    const T* base_ptr = static_cast<const T*>(a.logits) + row * a.stride;
    const int off = int(reinterpret_cast<uintptr_t>(base_ptr) / sizeof(T) % VE);
    const int q0 = off > 0 ? 1 : 0, whole = (off + a.vocab) / VE;
    const int per = (max(whole - q0, 0) + a.cluster - 1) / a.cluster;
    Sampler<T> s{a, sh, {base_ptr, off, a.vocab, q0 + rank * per, min(whole, q0 + (rank + 1) * per),
                         rank == a.cluster - 1}, rank, {}, 0};
    if (a.cluster > 1) cluster_arrive();  // waited for below, before the first store to another block

    const float temp = a.temperature ? a.temperature[row] : 1.f;
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    const float raw_min_p = a.min_p ? a.min_p[row] : 0.f;
    const float min_p = fminf(raw_min_p, 1.f);
    const float u = a.uniform[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool greedy = temp <= 0.f;
    const bool by_k = top_k > 0 && top_k < a.vocab;
    const bool by_p = top_p < 1.f;
    const bool by_min = min_p > 0.f;
    // the last kept token, whose place is counted: sums of weights near the unit, rounded
    // together or one by one, do not tell the last of several apart
    const bool by_last = u >= 1.f;

    // ---- the largest logit, and the largest of every thread's elements ----
    // A NaN stays the largest, so one look at the end finds it (and a +inf).
    float m = -INFINITY;
    for_each<4>(s.part, a.dev_status, [&](float z, int) { m = max_nan(m, z); });
    sh.group[tid] = m;
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = max_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    if ((tid & 31) == 0) sh.warp_max[tid >> 5] = wm;
    if (tid == 0) sh.my_bound = -INFINITY;
    __syncthreads();
    // top-k: each block's j-th largest group maximum, j = ceil(k / blocks); at least k
    // elements of the row are as large as the smallest of these
    const bool heads_k = by_k && top_k <= kMaxHeads && !greedy;
    if (heads_k) {
        const int j = (top_k + a.cluster - 1) / a.cluster;
        int groups = 64;  // of neighbouring threads: larger groups bound less tightly but rank faster
        while (groups < 2 * j && groups < kThreads) groups *= 2;
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
    s.barrier();
    float row_max = -INFINITY, bound = INFINITY;
    for (int c = 0; c < a.cluster; ++c) {
        row_max = max_nan(row_max, sh.row_max[c]);
        bound = fminf(bound, sh.bound[c]);
    }
    const bool bad_row = !(row_max < INFINITY) || row_max == -INFINITY || !(temp == temp) || !(top_p == top_p) ||
                         !(u == u) || !(raw_min_p == raw_min_p);
    if (bad_row) {  // the same in every block; nobody has to read another's memory any more
        if (rank == 0 && tid == 0) {
            s.write(row, -1, __uint_as_float(0x7fc00000u));
            report(a.dev_status, VCE_DEVSTATUS_BAD_ROW);
        }
        return;
    }
    s.sc = make_scale(row_max, temp);
    const Scale sc = s.sc;

    if (greedy) {
        if (tid == 0) sh.argmax = 0xffffffffu;
        __syncthreads();
        uint32_t first = 0xffffffffu;
        for_each<2>(s.part, a.dev_status, [&](float z, int i) {
            if (z == row_max && uint32_t(i) < first) first = uint32_t(i);
        });
        if (first != 0xffffffffu) atomicMin(&sh.argmax, first);
        s.barrier();
        if (rank == 0 && tid == 0) {
            uint32_t best = 0xffffffffu;
            for (int c = 0; c < a.cluster; ++c) best = min(best, remote(&sh.argmax, c));
            s.write(row, best, 0.f);
        }
        s.barrier();  // nobody leaves while its shared memory is read
        return;
    }

    bool exact = true;
    uint64_t least = 0;  // min-p's least weight
    if (by_min) {
        least = uint64_t(1) << a.q_bits;
        if (min_p < 1.f) {
            const uint64_t f = floor_product(min_p, least, &exact);
            least = exact ? f : f + 1;
        }
    }
    const bool heads_min = by_min && !by_p;
    uint64_t key = 0, weight_drawn = 0, mass = 0, above = 0;
    int step = heads_k || heads_min ? kHeads : kTopK;
#pragma unroll 1
    for (;; ++step) {
        uint64_t target = 0, base = 0;
        uint32_t base_count = 0;
        Command cmd{0, ~0ull, -1, 0};
        if (step == kTopK) {
            // ---- weights of the whole row, summed by n ----
            for (int i = tid; i < kBins; i += kThreads) sh.mass[i] = 0, sh.count[i] = 0;
            // min-p (with top-p): whole bins above the border, and single weights next to it
            const int edge = by_min ? max(0, bin_of(fmaxf(a.least_log2, log2f(min_p))) - 2) : kBins;
            if (tid < kEdgeBins) sh.kept_minp[tid] = 0, sh.kept_n[tid] = 0;
            __syncthreads();
            uint32_t* const words = reinterpret_cast<uint32_t*>(sh.mass);  // low halves, then high ones
            for_pairs<1, 1>(s.part, a.dev_status, [&](float z0, float z1, int) {
                const Step2 st = step_of2(sc, make_float2(z0, z1));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (!((k ? st.p.y : st.p.x) < -a.least_log2)) continue;
                    const int bin = st.bin[k];
                    if (!VCE_BOUNDS(bin >= 0 && bin < kBins, a.dev_status)) continue;
                    const bool fine = bin < kFineBins;
                    const uint32_t coarse = (st.s[k] + (1u << (kCoarseBits - 1)) >> kCoarseBits) + kCoarseOffset;
                    const uint32_t x = fine ? st.s[k] : coarse;
                    atomicAdd(words + bin, x & ((1u << kHalfBits) - 1));
                    atomicAdd(words + kBins + bin, x >> kHalfBits);
                    if (fine || by_k || by_last) atomicAdd(&sh.count[bin], 1u);
                }
            });
            __syncthreads();
            {
                constexpr int kPer = (kBins + kThreads - 1) / kThreads;
                uint64_t v[kPer];
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const int i = tid + k * kThreads;
                    if (i >= kBins) break;
                    const uint64_t x = words[i] + (uint64_t(words[kBins + i]) << kHalfBits), c = sh.count[i];
                    v[k] = i < kFineBins ? x + (c << kFracBits) - (c << kBiasBits) : x << kCoarseBits;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (tid + k * kThreads < kBins) sh.mass[tid + k * kThreads] = v[k];
            }
            if (by_min) {  // the few elements of kEdgeBins bins
                const Wanted w = s.in_bin({0, ~0ull, edge + kEdgeBins / 2, 0});
                const float wide = 2.f / (kSteps * sc.ch);
                for_each<1>(s.part, a.dev_status, [&](float z, int) {
                    if (!(z >= w.z_lo - wide && z <= w.z_hi + wide)) return;
                    const float p = log2_weight(sc, z);
                    const int k = bin_of(p) - edge;
                    if (!(p > a.least_log2) || k < 0 || k >= kEdgeBins) return;
                    const uint64_t x = weight_of(sc, z, sh.table, a.q_bits);
                    if (x < least) return;
                    s.add_mass(&sh.kept_minp[k], x);
                    if (by_last) atomicAdd(&sh.kept_n[k], 1u);
                });
            }
            s.barrier();
            if (a.cluster > 1) {
                // Each block adds up all blocks' sums of its share of the bins and puts the
                // results into block 0 (whose sums of these bins nobody else reads).
                const int share = (kBins + a.cluster - 1) / a.cluster, end = min(kBins, (rank + 1) * share);
                for (int i = rank * share + tid; i < end; i += kThreads) {
                    uint64_t v[kMaxCluster];
                    uint32_t c[kMaxCluster];
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)  // all loads before the sums
                        if (r < a.cluster) v[r] = remote(&sh.mass[i], r), c[r] = remote(&sh.count[i], r);
                    uint64_t sum = 0;
                    uint32_t n = 0;
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)
                        if (r < a.cluster) sum += v[r], n += c[r];
                    put(&sh.mass[i], 0, sum);
                    put(&sh.count[i], 0, n);
                }
                s.barrier();
            }
            if (s.lead()) {
                constexpr int kPer = (kBins + kThreads - 1) / kThreads;
                prefix_sums<kPer>(sh.mass, kBins, sh.warp_sum, [&](int i) {
                    const uint64_t sum = sh.mass[i];
                    return sum ? scale_up(sum, i, sh.table, a.q_bits) : uint64_t(0);
                });
                if (by_k || by_last) prefix_sums<kPer>(sh.count, kBins, sh.warp_sum, [&](int i) { return sh.count[i]; });
                mass = sh.mass[kBins - 1];
                if (tid == 0) sh.n_kept = sh.count[kBins - 1];
                cmd.flag = by_k && sh.count[kBins - 1] > uint32_t(top_k);  // the k-th has a weight
                if (by_min) {
                    above = edge ? sh.mass[edge - 1] : 0;
                    uint32_t n_above = edge ? sh.count[edge - 1] : 0;
                    for (int k = 0; k < kEdgeBins; ++k) {  // the last bin with a kept weight decides
                        uint64_t kept = 0;
                        for (int c = 0; c < a.cluster; ++c) {
                            kept += remote(&sh.kept_minp[k], c);
                            n_above += remote(&sh.kept_n[k], c);
                        }
                        const int bin = edge + k;
                        if (kept) above = min((bin ? sh.mass[bin - 1] : 0) + kept, sh.mass[bin]);
                    }
                    if (tid == 0) sh.n_above = n_above;
                }
            }
            if (by_k && !s.tell(cmd).flag) continue;
            if (!by_k) continue;
            target = uint64_t(top_k);
        } else if (step == kTopP) {
            if (!by_p) continue;
            target = floor_product(fmaxf(top_p, 0.f), mass, &exact);
            target += exact ? 0 : 1;
            if (target == 0) target = 1;
        } else if (step == kDraw) {
            if (by_min && above < mass) mass = above;
            if (by_last) {
                __syncthreads();
                target = by_min ? min(sh.n_kept, sh.n_above) : sh.n_kept;
            } else {
                target = floor_product(fmaxf(u, 0.f), mass, &exact) + 1;
            }
        }
        const bool by_count = step == kTopK || (step == kDraw && by_last);
        // ---- the border's bin, told to all ----
        Wanted w{0.f, row_max, heads_min ? fmaxf(a.least_log2, log2f(min_p) - 0.01f) : a.least_log2, cmd};
        w.z_lo = heads_k ? bound : sc.m + (w.p_least - 0.1f) / sc.ch - fabsf(sc.m) * 0x1p-21f;
        if (step != kHeads) {
            if (s.lead()) {
                cmd.bin = min(by_count ? first_at_least(sh.count, kBins, uint32_t(target))
                                       : first_at_least(sh.mass, kBins, target),
                              kBins - 1);
                if (cmd.bin > 0) base = sh.mass[cmd.bin - 1], base_count = sh.count[cmd.bin - 1];
            }
            w = s.in_bin(s.tell(cmd));
        }
        // ---- its elements, collected and sorted ----
        // Keys have 52 bits and differ, and a division leaves at most 2^-11 of their range
        // (one key at last): five levels at most.
#pragma unroll 1
        for (int level = 0; level < 8; ++level) {
            s.collect(w);
            cmd = w.cmd;
            if (s.lead()) {
                int n;
                cmd.flag = s.join_lists(n);
                if (cmd.flag) {
                    sort_list(sh.list, n, sh.sums);
                    auto weight = [&](int i) {
                        return weight_of(sc, key_logit(sh.list[i]), sh.table, a.q_bits) + (i == 0 ? base : 0);
                    };
                    if (n <= kThreads) prefix_sums<1>(sh.sums, n, sh.warp_sum, weight);
                    else prefix_sums<kCap / kThreads>(sh.sums, n, sh.warp_sum, weight);
                    int at;
                    if (by_count) {
                        at = int(target - base_count) - 1;
                    } else {
                        if (step == kHeads) {
                            if (by_k && top_k < n) n = top_k;
                            mass = sh.sums[n - 1];
                            if (by_p) {
                                target = floor_product(fmaxf(top_p, 0.f), mass, &exact);
                                target += exact ? 0 : 1;
                                n = first_at_least(sh.sums, n, target ? target : uint64_t(1)) + 1;
                            }
                            if (by_min) {  // weights descend: the first that is too small ends the head
                                __syncthreads();
                                if (tid == 0) sh.found = uint32_t(n);
                                __syncthreads();
                                for (int i = tid; i < n; i += kThreads)
                                    if (sh.sums[i] - (i ? sh.sums[i - 1] : 0) < least) atomicMin(&sh.found, uint32_t(i));
                                __syncthreads();
                                n = max(1, int(sh.found));
                            }
                            mass = sh.sums[n - 1];
                            target = by_last ? mass : floor_product(fmaxf(u, 0.f), mass, &exact) + 1;
                        }
                        at = first_at_least(sh.sums, n, target);
                    }
                    at = max(0, min(at, n - 1));
                    key = sh.list[at];
                    weight_drawn = sh.sums[at] - (at ? sh.sums[at - 1] : base);
                    // (never past the border's bin: weights rounded one by one can sum to more than
                    // the bin's, which was rounded once, and the draw would look behind the bin)
                    if (step == kTopK || step == kTopP) {
                        mass = min(sh.sums[at], sh.mass[cmd.bin]);
                        if (tid == 0) sh.n_kept = base_count + at + 1;
                    }
                }
            }
            cmd = s.tell(cmd);
            if (cmd.flag || step == kHeads) break;
            Sampler<T> copy = s;  // its address is taken there, not here
            copy.divide(cmd, by_count, target, base, base_count);
            s.turn = copy.turn;
            w = s.in_bin(cmd);
        }
        if (step == kDraw || (step == kHeads && cmd.flag)) break;  // heads that are too many: by masses
    }
    if (s.lead() && tid == 0) s.finish(row, key, weight_drawn, mass, temp);
    s.barrier();  // nobody leaves while its shared memory is read
}

}  // namespace

vce_status launch_ce_sample(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                            const float* uniform, const float* temperature, const int* top_k, const float* top_p,
                            const float* min_p, int64_t* token, float* logprob, int* dev_status, cudaStream_t s,
                            const DeviceInfo& dev) {
    if (n == 0) return VCE_OK;
    SampleArgs a{logits, n, stride, int(vocab), uniform, temperature, top_p, min_p, top_k, token, logprob, 1, 0,
                 0.f, dev_status};
    int bits = 0;
    while ((int64_t(1) << bits) < vocab) ++bits;
    a.q_bits = 63 - bits < 44 ? 63 - bits : 44;
    // half a unit, and 2^-10 for the rounding of a log2_weight (below 2^-16): whatever is counted
    // has a weight that is not 0 after its rounding either
    a.least_log2 = -float(a.q_bits + 1) + 0x1p-10f;
    // As many blocks per row as fill the SMs once, each with a part worth a block.  (Filled
    // twice, 256 x 128256 rows took 171 -> 144 us where a few rows need several borders, but
    // 108 -> 135 us where all are alike.)
    while (a.cluster < kMaxCluster &&
           (vocab > int64_t(a.cluster) * (kMaxPart - 64) ||
            (n * a.cluster * 2 <= 2 * dev.num_sms && vocab / (a.cluster * 2) >= 4 * kThreads)))
        a.cluster *= 2;
    if (n * a.cluster > 0x7fffffff) return VCE_ERR_INVALID_ARG;
    auto kernel = dtype == VCE_BF16 ? ce_sample_kernel<__nv_bfloat16> : ce_sample_kernel<float>;
    static std::mutex mu;
    static bool ready[64][2];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev.ordinal][dtype == VCE_BF16]) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Shared))) !=
                cudaSuccess)
                return VCE_ERR_CUDA;
            ready[dev.ordinal][dtype == VCE_BF16] = true;
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(n * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(a.cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
