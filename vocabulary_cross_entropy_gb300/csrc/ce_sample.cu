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
// 44 and leaves room for the sum of a row.  Integer sums are exact in any order: the
// row is split over threads and blocks freely, and atomics change nothing.
//
// A row never gets sorted as a whole:
//   heads  (top-k up to kMaxHeads, or min-p without top-p): a bound is found below
//          which nothing survives - the k-th largest of the maxima of disjoint groups
//          of elements, or min-p's own - and what lies above it, a little more than the
//          head, is collected and sorted in shared memory.
//   masses (otherwise): for every n the number of elements and the sum of their s are
//          collected, three 32-bit atomics each; n is ordered by construction and the
//          scaling by 2^(n / 64) happens once per n.  A border is located among the
//          prefix sums of the masses, and only the elements of that one n are collected
//          and sorted.  Too many of them are divided again by the bits of (logit, index).
// The logits are read once from HBM; the later passes find them in L2.
//
// A row is shared by a cluster of blocks (one when there are rows enough).  Block 0 joins
// the others' results, which it reads from their shared memory, and decides; the others
// read its decision.

#include "vce_internal.cuh"
#include "sm100_ptx.cuh"

#include <math.h>
#include <mutex>

namespace vce {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
#ifndef X_U
#define X_U 1
#endif
#ifndef X_FILL
#define X_FILL 2
#endif
constexpr int kSteps = 64;            // values of n per octave
constexpr int kBins = 46 * kSteps;    // 46 octaves of n, from 0 down
constexpr float kLeastLog2 = -45.9f;  // below it a weight is 0 (Q <= 44)
constexpr int kFracBits = 36;         // of s
constexpr int kBiasBits = 29;         // s - 2^36 is above -2^29 and below 2^29
constexpr int kHalfBits = 15;         // it is summed in two halves, which 2^17 elements cannot overflow
constexpr int kMaxPart = 1 << 17;     // elements per block
constexpr int kCap = 2048;          // collected elements; also sub-bins of a divided bin
constexpr int kCapBits = 11;
constexpr int kMaxHeads = 256;      // top-k of the collecting path
constexpr int kIndexBits = 20;      // vocabulary of at most 2^20
constexpr int kMaxCluster = 8;

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
    int* dev_status;
};

// What block 0 tells the others.
struct Command {
    uint64_t lo, hi;  // range of (logit, index) keys
    int bin, flag;
};

struct Shared {
    uint64_t mass[kBins];  // two 32-bit sums, then the sum of s, then (block 0) inclusive prefix sums of masses
    uint32_t count[kBins];
    uint64_t list[kCap];   // collected keys; masses of sub-bins
    uint64_t sums[kCap];   // inclusive prefix sums of the sorted list; counts of sub-bins
    uint64_t table[kSteps];
    uint64_t warp_sum[kWarps], warp_sum2[kWarps];
    float group[kThreads];
    float row_max[kMaxCluster], bound[kMaxCluster];  // a block writes its own slot, once
    int bad[kMaxCluster];
    Command cmd[2];  // consecutive commands take turns: a late reader finds its own intact
    uint64_t min_key, max_key, kept_minp;
    uint32_t n_list, found, argmax;
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

// The element's n (as the bin -n) and s of a log2_weight above kLeastLog2.
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

// round(2^Q 2^(-bin / 64) sum / 2^36) for a sum of s below 2^57
__device__ __forceinline__ uint64_t scale_up(uint64_t sum, int bin, const uint64_t* table, int q_bits) {
    const int n = -bin;
    const uint64_t t = table[n & (kSteps - 1)];                       // 63 fractional bits
    const int shift = 63 + kFracBits - q_bits - (n >> 6);             // 55 .. 102
    const uint64_t hi = __umul64hi(sum, t), lo = sum * t;
    uint64_t q;  // twice the value, rounded down
    if (shift - 1 < 64) q = hi << (65 - shift) | lo >> (shift - 1);
    else q = hi >> (shift - 65);
    return (q + 1) >> 1;
}

__device__ __forceinline__ uint64_t weight_of(const Scale& s, float z, const uint64_t* table, int q_bits) {
    const Step st = step_of(s, z);
    return scale_up((uint64_t(1) << kFracBits) + int64_t(st.g), st.bin, table, q_bits);
}

// floor(x y) for a float 0 <= x < 1 and y < 2^63; ``*exact`` tells whether nothing was cut off
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
// q holds elements q VE - off ...; the first and the last may reach past the row.
template <typename T>
struct Part {
    const T* row;
    int off, vocab;
    int q0, q1;
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

// fn(logit, index) for every element of the block's part, U vectors in flight per thread.
// The vectors that lie in the row as a whole come first, then the elements of the two
// that may not.
template <int U, typename T, typename F>
__device__ __forceinline__ void for_each(const Part<T>& p, int* dev_status, F fn) {
    constexpr int VE = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int head = p.off > 0 ? 1 : 0, whole = (p.off + p.vocab) / VE;  // whole vectors: [head, whole)
    const int end = min(p.q1, whole);
    for (int q = max(p.q0, head) + tid; q < end; q += U * kThreads) {
        const T* at = p.row + (q * VE - p.off);
        uint4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (q + k * kThreads < end && VCE_BOUNDS(aligned16(at), dev_status))
                v[k] = __ldg(reinterpret_cast<const uint4*>(at + k * kThreads * VE));
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (q + k * kThreads >= end) break;
            const int i = (q + k * kThreads) * VE - p.off;
#pragma unroll
            for (int e = 0; e < VE; ++e) fn(element<T>(v[k], e), i + e);
        }
    }
    // the first vector's elements, then those behind the whole vectors
    const int first = head && p.q0 == 0 && p.q1 > 0 ? min(VE - p.off, p.vocab) : 0;
    const int tail0 = max(whole * VE - p.off, head ? VE - p.off : 0);
    const int last = p.q1 > p.q0 && p.q1 * VE - p.off >= p.vocab ? max(p.vocab - tail0, 0) : 0;
    if (tid < first + last) {
        const int i = tid < first ? tid : tail0 + tid - first;
        fn(one(p.row + i), i);
    }
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

__device__ __forceinline__ void row_barrier(int cluster) {
    if (cluster == 1) __syncthreads();
    else cluster_sync();
}

// Inclusive prefix sums of a[0 .. n) in place (n at most 6 x kThreads); every thread calls.
template <typename T>
__device__ __forceinline__ void prefix_sums(T* a, int n, uint64_t* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (n + kThreads - 1) / kThreads;
    const int i0 = int(threadIdx.x) * per;
    uint64_t s = 0;
    for (int k = 0; k < per; ++k)
        if (i0 + k < n) s += a[i0 + k];
    uint64_t t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += x;
    }
    if (lane == 31) warp_sum[warp] = t;
    __syncthreads();
    uint64_t before = t - s;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int k = 0; k < per; ++k)
        if (i0 + k < n) {
            before += a[i0 + k];
            a[i0 + k] = T(before);
        }
    __syncthreads();
}

// Sorts list[0 .. n), n <= kCap, descending (all keys differ); ``tmp`` is scratch.
__device__ __forceinline__ void sort_list(uint64_t* list, int n, uint64_t* tmp) {
    const int t = threadIdx.x;
    if (n <= 128) {  // each key counts those before it
        if (t < n) {
            const uint64_t k = list[t];
            int r = 0;
            for (int j = 0; j < n; ++j) r += list[j] > k;
            tmp[r] = k;
        }
        __syncthreads();
        if (t < n) list[t] = tmp[t];
        __syncthreads();
        return;
    }
    int size = 256;
    while (size < n) size *= 2;
    for (int i = n + t; i < size; i += kThreads) list[i] = 0;  // after every key
    __syncthreads();
    for (int len = 2; len <= size; len *= 2)
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

    // Block 0's command, the same in every block: a barrier, after which all read it.  A slot
    // is written again two commands later, behind a barrier that its readers have passed.
    __device__ __forceinline__ Command tell(const Command& c) {
        Command* slot = &sh.cmd[turn & 1];
        ++turn;
        if (lead() && threadIdx.x == 0) *slot = c;
        barrier();
        if (a.cluster == 1) return *slot;
        return {remote(&slot->lo, 0), remote(&slot->hi, 0), remote(&slot->bin, 0), remote(&slot->flag, 0)};
    }

    __device__ __forceinline__ bool lead() const { return rank == 0; }
    __device__ __forceinline__ void barrier() const { row_barrier(a.cluster); }

    // Collects the keys of the elements that ``take`` accepts (its own part); all threads.
    template <typename F>
    __device__ __forceinline__ void collect(F take) {
        if (threadIdx.x == 0) sh.n_list = 0;
        __syncthreads();
        for_each<4>(part, a.dev_status, [&](float z, int i) {
            if (!take(z, i)) return;
            const uint32_t at = atomicAdd(&sh.n_list, 1u);
            if (at < kCap) sh.list[at] = key_of(z, i);
        });
    }

    // Block 0, after a barrier: the others' lists behind its own.  False when they
    // are too many.
    __device__ __forceinline__ bool join_lists(int& n) {
        uint32_t total = 0;
        for (int c = 0; c < a.cluster; ++c) total += c == 0 ? sh.n_list : remote(&sh.n_list, c);
        if (total > kCap) return false;
        uint32_t at = sh.n_list;
        for (int c = 1; c < a.cluster; ++c) {
            const uint32_t m = remote(&sh.n_list, c);
            for (uint32_t i = threadIdx.x; i < m; i += kThreads) sh.list[at + i] = remote(&sh.list[i], c);
            at += m;
        }
        n = int(total);
        __syncthreads();
        return true;
    }

    // Block 0: sorts the list and makes sh.sums its inclusive prefix sums from ``base``.
    __device__ __forceinline__ void sort_and_sum(int n, uint64_t base) {
        sort_list(sh.list, n, sh.sums);
        for (int i = threadIdx.x; i < n; i += kThreads)
            sh.sums[i] = weight_of(sc, key_logit(sh.list[i]), sh.table, a.q_bits) + (i == 0 ? base : 0);
        __syncthreads();
        prefix_sums(sh.sums, n, sh.warp_sum);
    }

    // Block 0: the first i < n with s[i] >= target (n when there is none).
    template <typename V>
    __device__ __forceinline__ int first_at_least(const V* s, int n, V target) {
        __syncthreads();
        if (threadIdx.x == 0) sh.found = uint32_t(n);
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads)
            if (s[i] >= target && (i == 0 || s[i - 1] < target)) sh.found = uint32_t(i);
        __syncthreads();
        return int(sh.found);
    }

    __device__ __forceinline__ void add_mass(uint64_t* at, uint64_t w) {
        atomicAdd(reinterpret_cast<unsigned long long*>(at), static_cast<unsigned long long>(w));
    }

    // Sum over the block of one value per thread; valid in thread 0.
    __device__ __forceinline__ uint64_t block_sum(uint64_t v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) == 0) sh.warp_sum2[threadIdx.x >> 5] = v;
        __syncthreads();
        uint64_t t = 0;
        if (threadIdx.x == 0)
            for (int w = 0; w < kWarps; ++w) t += sh.warp_sum2[w];
        __syncthreads();
        return t;
    }

    // The elements of ``cmd``'s bin and key range, whose logits lie between z_lo and z_hi.
    struct InBin {
        Scale s;
        float z_lo, z_hi;
        int bin;
        uint64_t lo, hi;
        __device__ __forceinline__ bool operator()(float z, int i) const {
            if (!(z >= z_lo && z <= z_hi)) return false;
            const float p = log2_weight(s, z);
            if (!(p > kLeastLog2) || bin_of(p) != bin) return false;
            const uint64_t k = key_of(z, i);
            return k >= lo && k <= hi;
        }
    };
    __device__ __forceinline__ InBin in_bin(const Command& cmd) const {
        // the bounds are generous; the bin itself decides
        const float far = (float(cmd.bin) + 0.75f) / (kSteps * sc.ch), near = (float(cmd.bin) - 0.75f) / (kSteps * sc.ch);
        const float slack = fabsf(sc.m) * 0x1p-21f;
        return {sc, sc.m - far - slack, sc.m - near + slack, cmd.bin, cmd.lo, cmd.hi};
    }

    // A range that holds more elements than a list: its keys divided into kCap ranges of
    // equal width, of which the one with the target is the new range.  ``base`` and
    // ``base_count`` become what lies before it.  Rare, and kept out of the common code.
    __device__ __noinline__ void divide(Command& cmd, bool by_count, uint64_t target, uint64_t& base,
                                        uint32_t& base_count) {
        const InBin mine = in_bin(cmd);
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
            prefix_sums(sh.list, kCap, sh.warp_sum);
            prefix_sums(sh.sums, kCap, sh.warp_sum);
            const int b = min(by_count ? first_at_least(sh.sums, kCap, target - base_count)
                                       : first_at_least(sh.list, kCap, target > base ? target - base : 1),
                              kCap - 1);
            if (b > 0) base += sh.list[b - 1], base_count += uint32_t(sh.sums[b - 1]);
            const uint64_t width = (uint64_t(1) << shift) - 1;
            cmd.hi = h - (uint64_t(b) << shift);
            cmd.lo = cmd.hi - l > width ? cmd.hi - width : l;
        }
        cmd = tell(cmd);
    }

    // Finds the first element, in order, at which the cumulated weight (or, by_count, the
    // number of elements) reaches ``target``.  All blocks call; the results are valid in
    // block 0: the element's key and the cumulated weight up to and with it.  ``target`` is
    // within the total.
    __device__ __forceinline__ void locate(bool by_count, uint64_t target, uint64_t& key, uint64_t& upto) {
        uint64_t base = 0;
        uint32_t base_count = 0;
        Command cmd{0, ~0ull, 0, 0};
        if (lead()) {
            cmd.bin = min(by_count ? first_at_least(sh.count, kBins, uint32_t(target))
                                   : first_at_least(sh.mass, kBins, target),
                          kBins - 1);
            if (cmd.bin > 0) base = sh.mass[cmd.bin - 1], base_count = sh.count[cmd.bin - 1];
        }
        cmd = tell(cmd);
        // Keys have 52 bits and differ, and a division leaves at most 2^-11 of their range
        // (one key at last): five levels at most.
        for (int level = 0; level < 8; ++level) {
            collect(in_bin(cmd));
            barrier();
            if (lead()) {
                int n;
                cmd.flag = join_lists(n);
                if (cmd.flag) {
                    sort_and_sum(n, base);
                    int at = by_count ? int(target - base_count) - 1 : first_at_least(sh.sums, n, target);
                    at = max(0, min(at, n - 1));
                    key = sh.list[at];
                    upto = sh.sums[at];
                }
            }
            cmd = tell(cmd);
            if (cmd.flag) return;
            Sampler copy = *this;  // its address is taken there, not here
            copy.divide(cmd, by_count, target, base, base_count);
            turn = copy.turn;
        }
    }

    __device__ void write(int64_t row, int64_t token, float logprob) {
        a.token[row] = token;
        if (a.logprob) a.logprob[row] = logprob;
    }

    // Block 0, thread 0: the drawn token and the logarithm of its share of the mass.
    __device__ void finish(int64_t row, uint64_t key, uint64_t mass, float t) {
        const float z = key_logit(key);
        const uint64_t w = weight_of(sc, z, sh.table, a.q_bits);
        float lp;
        if (w > mass / 2) lp = log1pf(-__ull2float_rn(mass - w) / __ull2float_rn(mass));
        else lp = (z - sc.m) / fminf(fmaxf(t, 1e-30f), 1e30f) - logf(ldexpf(__ull2float_rn(mass), -a.q_bits));
        write(row, key_index(key), lp);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) ce_sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const int tid = threadIdx.x;
    const int rank = a.cluster == 1 ? 0 : int(cluster_ctarank());
    const int64_t row = int64_t(blockIdx.x) / a.cluster;
    if (tid < kSteps) sh.table[tid] = kExp2Table[tid];

    constexpr int VE = 16 / sizeof(T);
    const T* base = static_cast<const T*>(a.logits) + row * a.stride;
    const int off = int(reinterpret_cast<uintptr_t>(base) / sizeof(T) % VE);
    const int vectors = (off + a.vocab + VE - 1) / VE;
    const int per = (vectors + a.cluster - 1) / a.cluster;
    Sampler<T> s{a, sh, {base, off, a.vocab, rank * per, min(vectors, (rank + 1) * per)}, rank, {}, 0};

    const float temp = a.temperature ? a.temperature[row] : 1.f;
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? fminf(a.min_p[row], 1.f) : 0.f;
    const float u = a.uniform[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool greedy = temp <= 0.f;
    const bool by_k = top_k > 0 && top_k < a.vocab;
    const bool by_p = top_p < 1.f;
    const bool by_min = min_p > 0.f;

    // ---- the largest logit, and the largest of every thread's elements ----
    float m = -INFINITY;
    for_each<4>(s.part, a.dev_status, [&](float z, int) { m = max_nan(m, z); });
    const bool bad = !(m < INFINITY);  // a NaN or +inf among them
    sh.group[tid] = m;
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    if ((tid & 31) == 0) sh.warp_sum[tid >> 5] = __float_as_uint(wm);
    const bool any_bad = __syncthreads_or(bad);
    // top-k: each block's j-th largest group maximum, j = ceil(k / blocks); at least k
    // elements of the row are as large as the smallest of these
    const int j = (top_k + a.cluster - 1) / a.cluster;
    const bool heads_k = by_k && top_k <= kMaxHeads;
    if (heads_k) {
        int groups = 64;  // of neighbouring threads: larger groups bound less tightly but rank faster
        while (groups < 4 * j && groups < kThreads) groups *= 2;
        const int width = kThreads / groups;
        float g = -INFINITY;
        if (tid < groups)
            for (int i = 0; i < width; ++i) g = fmaxf(g, sh.group[tid * width + i]);
        __syncthreads();
        if (tid < groups) sh.group[tid] = g;
        __syncthreads();
        if (tid < groups) {
            int before = 0;
            for (int i = 0; i < groups; ++i) before += sh.group[i] > g || (sh.group[i] == g && i < tid);
            if (before == j - 1) sh.bound[rank] = g;
        }
    }
    if (tid == 0) {
        float r = -INFINITY;
        for (int w = 0; w < kWarps; ++w) r = fmaxf(r, __uint_as_float(uint32_t(sh.warp_sum[w])));
        sh.row_max[rank] = r;
        sh.bad[rank] = any_bad;
    }
    s.barrier();
    float row_max = -INFINITY, bound = INFINITY;
    bool row_bad = !(temp == temp) || !(top_p == top_p) || !(u == u) || (a.min_p && !(a.min_p[row] == a.min_p[row]));
    for (int c = 0; c < a.cluster; ++c) {
        row_max = fmaxf(row_max, remote(&sh.row_max[c], c));
        row_bad |= remote(&sh.bad[c], c) != 0;
        if (heads_k) bound = fminf(bound, remote(&sh.bound[c], c));
    }
    if (row_bad || row_max == -INFINITY) {  // the same in every block
        if (rank == 0 && tid == 0) {
            s.write(row, -1, __uint_as_float(0x7fc00000u));
            report(a.dev_status, VCE_DEVSTATUS_BAD_ROW);
        }
        s.barrier();  // nobody leaves while its shared memory is read
        return;
    }
    s.sc = make_scale(row_max, temp);
    const Scale sc = s.sc;
    const uint64_t least = by_min ? [&] {
        bool exact;
        if (min_p >= 1.f) return uint64_t(1) << a.q_bits;
        const uint64_t f = floor_product(min_p, uint64_t(1) << a.q_bits, &exact);
        return exact ? f : f + 1;
    }() : 0;

    if (greedy) {
        if (tid == 0) sh.argmax = 0xffffffffu;
        __syncthreads();
        uint32_t first = 0xffffffffu;
        for_each<4>(s.part, a.dev_status, [&](float z, int i) {
            if (z == row_max && uint32_t(i) < first) first = uint32_t(i);
        });
        if (first != 0xffffffffu) atomicMin(&sh.argmax, first);
        s.barrier();
        if (rank == 0 && tid == 0) {
            uint32_t best = 0xffffffffu;
            for (int c = 0; c < a.cluster; ++c) best = min(best, remote(&sh.argmax, c));
            s.write(row, best, 0.f);
        }
        s.barrier();
        return;
    }

    bool exact;
    Command cmd{0, 0, 0, 0};
    // ---- few survivors: collect them all ----
    const bool heads_min = by_min && !by_p;
    if (heads_k || heads_min) {
        const float p_least = heads_min ? fmaxf(kLeastLog2, log2f(min_p) - 0.01f) : kLeastLog2;
        const float z_least = heads_k ? bound : -INFINITY;
        s.collect([=](float z, int) { return z >= z_least && log2_weight(sc, z) > p_least; });
        s.barrier();
        if (s.lead()) {
            int n;
            const bool fits = s.join_lists(n);
            if (fits) {
                s.sort_and_sum(n, 0);
                if (by_k && top_k < n) n = top_k;
                int kept = n;
                if (by_p) {
                    uint64_t target = floor_product(fmaxf(top_p, 0.f), sh.sums[n - 1], &exact);
                    target += exact ? 0 : 1;
                    kept = s.first_at_least(sh.sums, n, target ? target : 1) + 1;
                }
                if (by_min) {  // weights descend: the first that is too small ends the head
                    __syncthreads();
                    if (tid == 0) sh.found = uint32_t(n);
                    __syncthreads();
                    for (int i = tid; i < n; i += kThreads) {
                        const uint64_t w = sh.sums[i] - (i ? sh.sums[i - 1] : 0);
                        if (w < least) atomicMin(&sh.found, uint32_t(i));
                    }
                    __syncthreads();
                    kept = min(kept, max(1, int(sh.found)));
                }
                const uint64_t mass = sh.sums[kept - 1];
                uint64_t target = u >= 1.f ? mass - 1 : floor_product(fmaxf(u, 0.f), mass, &exact);
                const int at = s.first_at_least(sh.sums, kept, target + 1);
                if (tid == 0) s.finish(row, sh.list[min(at, kept - 1)], mass, temp);
            }
            cmd.flag = fits;
        }
        if (s.tell(cmd).flag) {
            s.barrier();  // block 0's shared memory is still read
            return;
        }
    }

    // ---- weights of the whole row, summed by n ----
    for (int i = tid; i < kBins; i += kThreads) sh.mass[i] = 0, sh.count[i] = 0;
    __syncthreads();
    // min-p (with top-p): whole bins above the border, and single weights next to it
    const int edge = by_min ? max(0, bin_of(fmaxf(kLeastLog2, log2f(min_p))) - 2) : kBins;
    uint64_t above = 0;
    for_each<X_U>(s.part, a.dev_status, [&](float z, int) {
        if (!(log2_weight(sc, z) > kLeastLog2)) return;
        const Step st = step_of(sc, z);
        if (!VCE_BOUNDS(st.bin >= 0 && st.bin < kBins, a.dev_status)) return;
        const uint32_t x = uint32_t(st.g + (1 << kBiasBits));
        uint32_t* at = reinterpret_cast<uint32_t*>(&sh.mass[st.bin]);
        atomicAdd(at, x & ((1u << kHalfBits) - 1));
        atomicAdd(at + 1, x >> kHalfBits);
        atomicAdd(&sh.count[st.bin], 1u);
        if (st.bin >= edge && st.bin < edge + 5) {
            const uint64_t w = weight_of(sc, z, sh.table, a.q_bits);
            if (w >= least) above += w;
        }
    });
    if (by_min) {
        above = s.block_sum(above);
        if (tid == 0) sh.kept_minp = above;
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) {
        const uint64_t m2 = sh.mass[i], c = sh.count[i];
        sh.mass[i] = (c << kFracBits) - (c << kBiasBits) + (m2 & 0xffffffffu) + ((m2 >> 32) << kHalfBits);
    }
    s.barrier();
    uint64_t total = 0;
    if (s.lead()) {
        for (int i = tid; i < kBins; i += kThreads) {
            uint64_t sum = sh.mass[i];
            uint32_t c = sh.count[i];
            for (int r = 1; r < a.cluster; ++r) sum += remote(&sh.mass[i], r), c += remote(&sh.count[i], r);
            sh.mass[i] = c ? scale_up(sum, i, sh.table, a.q_bits) : 0;
            sh.count[i] = c;
        }
        __syncthreads();
        prefix_sums(sh.mass, kBins, sh.warp_sum);
        if (by_k) {
            prefix_sums(sh.count, kBins, sh.warp_sum);
            cmd.flag = sh.count[kBins - 1] > uint32_t(top_k);  // the k-th has a weight
        }
        total = sh.mass[kBins - 1];
        if (by_min) {
            above = edge ? sh.mass[edge - 1] : 0;
            for (int c = 0; c < a.cluster; ++c) above += remote(&sh.kept_minp, c);
        }
    }
    // the border of top-k, then of top-p, then the draw: one after the other, each of
    // them within the mass that the one before left
    const bool cut = by_k && s.tell(cmd).flag;
    uint64_t key = 0, mass = total, upto = 0;
#pragma unroll 1
    for (int step = cut ? 0 : by_p ? 1 : 2; step < 3; ++step) {
        uint64_t target;
        if (step == 0) {
            target = uint64_t(top_k);
        } else if (step == 1) {
            if (!by_p) continue;
            target = floor_product(fmaxf(top_p, 0.f), mass, &exact);
            target += exact ? 0 : 1;
            if (target == 0) target = 1;
        } else {
            if (by_min && above < mass) mass = above;
            target = u >= 1.f ? mass : floor_product(fmaxf(u, 0.f), mass, &exact) + 1;
        }
        s.locate(step == 0, target, key, upto);
        if (step < 2) mass = upto;
    }
    if (s.lead() && tid == 0) s.finish(row, key, mass, temp);
    s.barrier();
}

}  // namespace

vce_status launch_ce_sample(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                            const float* uniform, const float* temperature, const int* top_k, const float* top_p,
                            const float* min_p, int64_t* token, float* logprob, int* dev_status, cudaStream_t s,
                            const DeviceInfo& dev) {
    if (n == 0) return VCE_OK;
    SampleArgs a{logits, n, stride, int(vocab), uniform, temperature, top_p, min_p, top_k, token, logprob, 1, 0,
                 dev_status};
    int bits = 0;
    while ((int64_t(1) << bits) < vocab) ++bits;
    a.q_bits = 63 - bits < 44 ? 63 - bits : 44;
    // As many blocks per row as fill the SMs twice, each with a part worth a block
    while (a.cluster < kMaxCluster &&
           (vocab > int64_t(a.cluster) * (kMaxPart - 64) ||
            (n * a.cluster * 2 <= X_FILL * dev.num_sms && vocab / (a.cluster * 2) >= 4 * kThreads)))
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
