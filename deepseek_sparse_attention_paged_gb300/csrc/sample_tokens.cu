// sample_tokens.cu -- the next token of every row of logits: temperature, top-k, top-p and min-p, then a draw
// with a given random number (sm_103a).
//
// Mathematics: w = 2^((z - max z) log2 e / temperature); order: larger z first, ties by index.  top-k keeps the
// first k; top-p those of them before which less than p of their mass lies; min-p those with w >= min_p.  The
// token is the least v with sum_{i <= v} w_i > u sum w over what is kept.
//
// Sums: a token must not depend on how a sum is split, and a border between two of 10^5 tokens is missed where sums
// are off by 10^-5 of a weight.  So a weight is formed to 2^-30 of itself (2^-35 for the largest, which count in every
// sum) and held as an integer, 2^46 about the largest: integer sums do not round, in any order, and u S and p M are
// compared exactly (24 x 64 bits).  1024 log2 w = n + f: one fused product leaves f with all the bits it needs
// (|f| <= 1/2), 2^(n / 1024) is a shift and a table of 1024 integers, 2^(f / 1024) a quadratic.  The fp64 unit would take ten
// times as long as the read of the row.
//
// A row is split over the CTAs of a cluster, each with a slice of it in shared memory: logits are read from global
// memory once.
//   * top-k up to 1024: the k-th largest of the maxima of all threads (or pairs of them) is a bound from below that few more
//     than k entries pass (with G maxima about -G ln(1 - k / G)).  Only the threads whose own maximum reaches it look at their
//     entries again; those that pass go to the first CTA, which does the rest alone.
//   * top-p without top-k: masses of 1024 bins of z (32 an octave of w) find the bin of the border; its entries
//     go to the first CTA, which finds the last one kept.  With that the masses say what each CTA keeps, and the one
//     that the random number falls to looks for the token in a second pass.
//     For bf16 the values themselves are the bins, and counts take the place of masses.
//   * where more entries than fit (2048) come together (ties, a temperature far above 1), or for a larger top-k:
//     bisection over the 32 bits of z, a pass over the slices each.
//
// Measured (calls in a captured graph): one row of 32000 (bf16) with top-k 50 and top-p 8.8 us, 64 of 131072 (fp32) with
// top-k, top-p and min-p, a setting each, 49 us, 300 of 100003 (bf16) with top-p alone 84 us, 256 of 131072 (fp32) with top-k 50
// and the probabilities written 64 us: 268 MB at 4.2 TB/s.  Bound: a few rows by the cluster's exchanges (launch, maxima, list,
// sums: about 1.2 us each) and by the slowest of eight CTAs; many rows with a top-k by the memory while all CTAs read and
// by latency while all select; top-p alone by forming a weight of 30 bits per entry (about 20 integer instructions) and by
// shared-memory atomics for the bins.
#include <float.h>

#include <algorithm>
#include <cstddef>

#include "dsa_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kMaxCtas = 8;
constexpr int kList = 2048;                    // entries that the first CTA takes in
constexpr int kMaxima = 2048;                  // that bound the k-th largest entry from below
constexpr int kFew = 128;                      // entries that are compared with one another
constexpr int kMaxTopK = 1024;
constexpr int kBins = 1024, kBinsPerOctave = 32;
constexpr int kSelectBins = 256;
// bf16 numbers from 2^-9 up to 2^7, of both signs, each a bin: 16 octaves of 128; in the middle one for all smaller ones
constexpr int kOddList = 3000;                 // entries of other values that are listed
constexpr int kSide = 16 * 128, kValueBins = 2 * kSide + 1, kFirstBits = (127 - 9) << 7;
constexpr int kOne = 46;                       // fraction bits of a weight
constexpr int kSingleRows = 64, kSingleVocab = 2048;   // where a CTA takes a row for itself
constexpr int kMaxSampleVocab = 1 << 18;       // sums of weights stay below 2^64
constexpr int kPowBits = 10;
constexpr int kMaxSmem = 227 * 1024;

// 2^(j / 1024) with kOne - 1 fraction bits, by the exponential series in 62-bit fixed point, and with 31.
struct PowTable {
    uint64_t fine[1 << kPowBits];
    uint32_t coarse[1 << kPowBits];
};
constexpr PowTable make_pow_table() {
    using u128 = unsigned __int128;
    PowTable t{};
    u128 ln2 = 0;                                            // sum 1 / (i 2^i)
    for (int i = 1; i < 80; ++i) ln2 += ((u128(1) << 100) >> i) / i;
    ln2 >>= 38;
    for (int j = 0; j < (1 << kPowBits); ++j) {
        const u128 x = (ln2 * j) >> kPowBits;
        u128 term = u128(1) << 62, sum = 0;
        for (int n = 1; term != 0; ++n) {
            sum += term;
            term = ((term * x) >> 62) / n;
        }
        t.fine[j] = static_cast<uint64_t>((sum + (u128(1) << (62 - kOne))) >> (63 - kOne));
        t.coarse[j] = static_cast<uint32_t>((sum + (u128(1) << 30)) >> 31);
    }
    return t;
}
__device__ const PowTable kPow = make_pow_table();

struct SampleArgs {
    const void* logits;
    int64_t ld;
    int V;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* tokens;
    float* probs;
    int64_t ld_probs;
    int ctas, slice;                           // CTAs of a row, entries of a CTA
    uint32_t region;                           // part of the list that a CTA has without a count beforehand
    int32_t* err;
};

template <int NT>
struct alignas(16) SampleShared {
    static constexpr int kStage = kBins;                       // (8 KB)
    static_assert(kStage >= 2 * kFew && kStage <= kList, "scratch");
    union {
        float maxima[NT == 1024 ? kMaxCtas * NT / 2 : kMaxima];   // of all CTAs (one of 1024 threads has its counts here)
        uint2 hist[kBins];                     // masses (low and high word)
        uint64_t stage[kStage];                // entries of this CTA on their way to the first one
        struct {
            uint64_t entry[kFew], mass[kFew];
        } few;
    };
    uint64_t list[kList];                      // first CTA: (order key of z, ~index)
    uint32_t pow[1 << kPowBits];
    uint2 sel_mass[kSelectBins];
    uint32_t sel_count[kSelectBins];
    uint64_t sel_value;
    uint64_t sum, limit;
    // written by all CTAs of the cluster
    float cta_max[kMaxCtas];
    int cta_index[kMaxCtas];
    uint32_t cta_count[kMaxCtas];
    uint64_t cta_sum[2][kMaxCtas];
    uint32_t cut_key;
    int cut_index;
    int bin;
    uint64_t bin_before, border_mass;
    // this CTA's
    uint64_t warp_sum[2][NT / 32];
    uint32_t warp_lo[NT / 32], warp_hi[NT / 32];
    float warp_max[NT / 32];
    uint32_t stage_count, quota;
    int found;
    double t_ln_min;                           // temperature ln min_p
    float rh, rl, zmin;
    float2 inv;
};

// ---------------------------------------------------------------- cluster

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_addr(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void put(void* p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void put(void* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t get(const void* p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t wide(uint2 h) { return (static_cast<uint64_t>(h.y) << 32) | h.x; }
__device__ __forceinline__ uint2 get2(const void* p, uint32_t rank) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote(p, rank)) : "memory");
    return v;
}
// ---------------------------------------------------------------- numbers

// Unsigned order of finite fp32 numbers and -infinity; -0 and 0 are one number.
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
    return (b & 0x80000000u) != 0u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) != 0u ? k & 0x7fffffffu : ~k);
}

// The largest logit and 1024 log2 e / t = rh + rl.
struct Scale {
    float top, rh, rl;
    int e0;                    // weights are held relative to 2^e0: e0 - 1 <= log2 e / t max z < e0
    bool wide;                 // log2 e / t max z past the range of `split`: relative to twice the largest weight
};
constexpr float kMagic = 12582912.0f;                        // 1.5 2^23: adding it rounds to whole numbers
constexpr int kMagicBits = 0x4b400000;
constexpr float kWide = 3900.0f;                             // |1024 y| stays below 2^22 down to weights of 2^-160
constexpr int kFine = 8;                                     // octaves below 2^e0 with the fine table

__device__ __forceinline__ Scale make_scale(float top, float rh, float rl) {
    const float y = top * rh * (1.0f / 1024.0f);             // infinite where rh overflowed: wide
    Scale c{top, rh, rl, 1, !(fabsf(y) < kWide)};
    // 1 more where rounding may have lost it (a scale of all weights)
    if (!c.wide) c.e0 = static_cast<int>(floorf(y + 0x1p-10f)) + 1;
    return c;
}

// shr and shl of more than 31 places give 0
__device__ __forceinline__ uint32_t shr(uint32_t v, int n) {
    uint32_t r;
    asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(n));
    return r;
}

// w 2^kOne = x 2^-shift, x of 46 bits, for log2 w = (n + f) / 1024, |f| <= 1 / 2
__device__ __forceinline__ uint64_t power_fine(int n, float f, int e0, int& shift) {
    // 2^(f / 1024) - 1 with 41 fraction bits: ln 2 / 1024 and ln^2 2 / 2 / 1024^2 times 2^41
    constexpr float c1 = 0.69314718055994531f * 0x1p31f, c2 = 0.24022650695910072f * 0x1p21f, c3 = 0.05550410866482158f * 0x1p11f;
    const int g = __float2int_rn(f * __fmaf_rn(f, __fmaf_rn(f, c3, c2), c1));
    const uint64_t p = kPow.fine[n & ((1 << kPowBits) - 1)];
    shift = e0 - 1 - (n >> kPowBits);
    return p + static_cast<uint64_t>((static_cast<int64_t>(static_cast<int>(p >> 15)) * g) >> 26);
}

// 1024 log2 of the weight relative to 2^e0 as n + f, n as it stands in the bits of a float past kMagic.  The product's
// rounding errors are those of f alone (2^-25 of 1/1024 octave), as n is taken from it before it is rounded.
__device__ __forceinline__ int split(float z, const Scale& c, float& f) {
    float e = 0.0f;
    if (c.wide) {                                            // z - max z, as a pair, in the place of z
        const float d = __fsub_rn(z, c.top);
        e = two_sum_err(z, -c.top, d);
        z = d;
    }
    const float t = __fmaf_rn(z, c.rh, kMagic);
    f = __fmaf_rn(z, c.rl, __fmaf_rn(z, c.rh, -__fsub_rn(t, kMagic)));
    if (c.wide) f = __fmaf_rn(e, c.rh, f);
    return __float_as_int(t);
}

// Mantissa (31 fraction bits, in [1, 2)) and exponent of the weight relative to 2^e0.
__device__ __forceinline__ uint32_t power(int bits, float f, const uint32_t* pow) {
    // 2^(f / 1024) - 1 with 32 fraction bits, rounded by the addition of kMagic
    constexpr float c1 = 0.69314718055994531f * 0x1p22f, c2 = 0.24022650695910072f * 0x1p12f;
    const int g = __float_as_int(__fmaf_rn(f, __fmaf_rn(f, c2, c1), kMagic)) - kMagicBits;
    const uint32_t p = pow[bits & ((1 << kPowBits) - 1)];
    // p g / 2^32 for unsigned p: the signed product counts p - 2^32
    return p + static_cast<uint32_t>(__mulhi(static_cast<int>(p), g) + g);
}
__device__ __forceinline__ int octave(int bits, const Scale& c) { return (bits >> kPowBits) - (kMagicBits >> kPowBits) - c.e0; }

// w 2^kOne / 2^e0 as a whole number, 0 below 2^-(kOne + 1)
__device__ __forceinline__ uint64_t weight(float z, const Scale& c, const uint32_t* pow) {
    float f;
    const int bits = split(z, c, f);
    const int i = octave(bits, c);                           // 2^i <= w < 2^(i + 1), i < 0
    if (i >= -kFine) {
        int shift;
        const uint64_t x = power_fine(bits - kMagicBits, f, c.e0, shift);
        return x >> shift;
    }
    const uint32_t m = power(bits, f, pow);
    const int left = i + kOne - 31;                          // of m
    // cut bits leave a 1 in the last place: as often too much as too little
    uint32_t w = shr(m, max(-left, 0));
    w |= min(w, 1u);
    return static_cast<uint64_t>(w) << max(left, 0);
}

// w / sum, from 1 / sum as a pair: rounded once
__device__ __forceinline__ float probability(float z, const Scale& c, const uint32_t* pow, float2 inv) {
    float f;
    const int bits = split(z, c, f);
    const int i = octave(bits, c);
    if (i < -160) return 0.0f;
    const uint32_t m = power(bits, f, pow);
    const float xh = static_cast<float>(m >> 8), xl = static_cast<float>(m & 0xffu) * 0x1p-8f;
    const float p = __fmaf_rn(xh, inv.x, __fmaf_rn(xh, inv.y, xl * inv.x));     // m / 2^8 / sum, at least 2^-41
    const int e = i + kOne - 31 + 8, first = max(e, -80);    // a subnormal number rounds once
    return p * __int_as_float((127 + first) << 23) * __int_as_float((127 + e - first) << 23);
}

// floor(a s), rounded up where `up` is set and it is not whole: a >= 0; saturates
__device__ __forceinline__ uint64_t scaled(float a, uint64_t s, bool up) {
    if (!(a > 0.0f)) return 0;
    const uint32_t b = __float_as_uint(a);
    const int ex = static_cast<int>(b >> 23);
    const uint64_t m = ex != 0 ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int right = 150 - max(ex, 1);                      // a = m 2^-right
    const uint64_t lo = m * s, hi = __umul64hi(m, s);
    if (right <= 0) return ~0ull;                            // a >= 2^23
    uint64_t out, rest;
    if (right < 64) {
        if ((hi >> right) != 0u) return ~0ull;
        out = (hi << (64 - right)) | (lo >> right);
        rest = lo & ((1ull << right) - 1);
    } else if (right < 128) {
        out = right == 64 ? hi : hi >> (right - 64);
        rest = lo | (right == 64 ? 0 : hi & ((1ull << (right - 64)) - 1));
    } else {
        out = 0;
        rest = hi | lo;
    }
    return out + (up && rest != 0 ? 1 : 0);
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// ---------------------------------------------------------------- the slice

// What is kept: z above `z`, and entries equal to it up to index `index`.
struct Cut {
    float z;
    int index;
    __device__ __forceinline__ bool keeps(float x, int v) const { return x > z || (x == z && v <= index); }
};

// NaN counts as -infinity, +infinity as the largest number of the type.
template <typename E>
__device__ __forceinline__ float largest() { return sizeof(E) == 4 ? FLT_MAX : __uint_as_float(0x7f7f0000u); }
__device__ __forceinline__ float clean(float z, float most) { return fminf(fmaxf(z, -INFINITY), most); }

__device__ __forceinline__ float bin_value(int bin) {
    const uint32_t bits = bin > kSide ? kFirstBits + (bin - kSide - 1) : 0x8000u | (kFirstBits + (kSide - 1 - bin));
    return __uint_as_float(bits << 16);
}

// 16 bytes of a row, entries outside [begin, end) -infinity.
template <typename E>
__device__ __forceinline__ uint4 load_group(const E* row, int v, int begin, int end) {
    constexpr int n = 16 / sizeof(E);
    if (v >= begin && v + n <= end) return __ldg(reinterpret_cast<const uint4*>(row + v));
    uint32_t w[4];
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v + i >= begin && v + i < end ? __ldg(reinterpret_cast<const uint32_t*>(row) + v + i) : 0xff800000u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = v + 2 * i + j;
                h[j] = k >= begin && k < end ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(row) + k)) : 0xff80u;
            }
            w[i] = h[0] | (h[1] << 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA's slice of a row: groups of 16 bytes on 16-byte boundaries, entries outside the slice -infinity.  Warp w has the
// groups [w per, (w + 1) per), its lanes one after the other: warps, steps and lanes follow the indices, and a thread
// reads only what it wrote itself.  kStaged: the slice lies in shared memory, read from global memory once.  Else every
// pass reads it from there, the first into L2.
// kDepth: groups that a thread loads together where it reads global memory (by the registers that the kernel has).
template <typename E, bool kStaged, int kDepth>
struct Slice {
    static constexpr int kGroup = 16 / sizeof(E);
    uint4* data;
    const E* row;
    float most;                                // values are cut to it: the type's largest, once it is known the row's
    int first;                                 // index of the first entry of group 0 (may lie before the slice)
    int begin, end;                            // indices of the slice
    int g0, g1;                                // groups of this warp
    int lane;

    __device__ __forceinline__ static void unpack(const uint4& r, float (&x)[kGroup]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
    __device__ __forceinline__ int steps() const { return (g1 - g0 + 31) / 32; }
    __device__ __forceinline__ int group_index(int g) const { return first + g * kGroup; }
    __device__ __forceinline__ uint4 raw(int g) const {
        if constexpr (kStaged) return data[g];
        else return load_group<E>(row, group_index(g), begin, end);
    }
    __device__ __forceinline__ void values(const uint4& r, float (&x)[kGroup]) const {
        unpack(r, x);
        if constexpr (!kStaged) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) x[i] = clean(x[i], most);
        }
    }
    // The first pass: the largest entry of this thread's, in kParts parts; f(group, its index) for each group as it lies in
    // memory.
    template <int kParts, typename F>
    __device__ __forceinline__ void take_in(float (&top)[kParts], F f) const {
        constexpr int kLoads = kDepth;
        static_assert(kGroup % kParts == 0, "parts");
#pragma unroll
        for (int i = 0; i < kParts; ++i) top[i] = -INFINITY;
        for (int g = g0 + lane; g < g1; g += 32 * kLoads) {
            uint4 r[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (g + 32 * i < g1) r[i] = load_group<E>(row, group_index(g + 32 * i), begin, end);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (g + 32 * i < g1) {
                    f(r[i], group_index(g + 32 * i));
                    float x[kGroup];
                    unpack(r[i], x);
                    if constexpr (kStaged) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < kGroup; ++e) x[e] = clean(x[e], most);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = sizeof(E) == 4 ? __float_as_uint(x[e % kGroup])
                                                  : (__float_as_uint(x[(2 * e) % kGroup]) >> 16) | __float_as_uint(x[(2 * e + 1) % kGroup]);
                        data[g + 32 * i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
#pragma unroll
                    for (int e = 0; e < kGroup; ++e) top[e % kParts] = fmaxf(top[e % kParts], x[e]);
                }
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) top[i] = fminf(top[i], most);
    }
    // entries of this lane's group of a step; -infinity past the warp's groups
    __device__ __forceinline__ int read(int step, float (&x)[kGroup]) const {
        const int g = g0 + step * 32 + lane;
        if (g < g1) {
            values(raw(g), x);
        } else {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) x[i] = -INFINITY;
        }
        return group_index(g);
    }
    // f(group, its index) for every group of this thread, as it lies in memory
    template <typename F>
    __device__ __forceinline__ void each_group(F f) const {
        constexpr int kLoads = kStaged ? 1 : kDepth;
        for (int g = g0 + lane; g < g1; g += 32 * kLoads) {
            uint4 r[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                if (g + 32 * j < g1) r[j] = raw(g + 32 * j);
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                if (g + 32 * j < g1) f(r[j], group_index(g + 32 * j));
        }
    }
    // f(z, index) for every entry of this thread
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        each_group([&](const uint4& r, int v) {
            float x[kGroup];
            values(r, x);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) f(x[i], v + i);
        });
    }
};

// ---------------------------------------------------------------- the first CTA's list

__device__ __forceinline__ uint64_t list_entry(float z, int v) { return (static_cast<uint64_t>(order_key(z)) << 32) | ~static_cast<uint32_t>(v); }
__device__ __forceinline__ float list_value(uint64_t e) { return key_value(static_cast<uint32_t>(e >> 32)); }
__device__ __forceinline__ int list_index(uint64_t e) { return static_cast<int>(~static_cast<uint32_t>(e)); }

// Sum over the block; all threads get it.  `slot` alternates between two calls in a row.
template <int NT>
__device__ __forceinline__ uint64_t block_sum64(SampleShared<NT>& s, uint64_t v, int slot) {
    v = warp_sum64(v);
    if ((threadIdx.x & 31) == 0) s.warp_sum[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t += s.warp_sum[slot][w];
    return t;
}

// Adds a 64-bit number to one in shared memory kept as two words (the exact sum, in any order).
__device__ __forceinline__ void add_wide(uint2* h, uint64_t w) {
    const uint32_t wl = static_cast<uint32_t>(w), old = atomicAdd(&h->x, wl);
    const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
    if (wh != 0u) atomicAdd(&h->y, wh);
}

// What a selection over the list goes by: from the largest z down by number or by mass, or from the lowest index up by mass.
enum Order { kByCount, kByMass, kByIndex };

// Entries list[0, n) that are `least` or more, in the given order: the one whose mass takes the sum from below `limit`
// to it or past it (the total reaches it).  By 256 bins of the range of values in turn.
template <int NT>
__device__ __noinline__ uint64_t select(SampleShared<NT>& s, int n, uint64_t least, Order order, uint64_t limit, const Scale c) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto value = [&](uint64_t e) { return order == kByIndex ? e << 32 : e; };
    uint32_t low = 0xffffffffu, high = 0;
    for (int i = tid; i < n; i += NT) {
        const uint64_t e = s.list[i];
        if (e < least) continue;
        const uint32_t v = static_cast<uint32_t>(value(e) >> 32);
        low = min(low, v);
        high = max(high, v);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    __syncthreads();
    if (lane == 0) {
        s.warp_lo[warp] = low;
        s.warp_hi[warp] = high;
    }
    if (tid < kSelectBins) {
        s.sel_mass[tid] = make_uint2(0u, 0u);
        s.sel_count[tid] = 0;
    }
    __syncthreads();
    for (int i = 0; i < NT / 32; ++i) {
        low = min(low, s.warp_lo[i]);
        high = max(high, s.warp_hi[i]);
    }
    uint64_t lo = static_cast<uint64_t>(low) << 32, range = (static_cast<uint64_t>(high - low) << 32) | 0xffffffffull;
    int shift = max(0, 64 - __clzll(static_cast<long long>(range)) - 8);
    for (;;) {
        for (int i = tid; i < n; i += NT) {
            const uint64_t e = s.list[i], v = value(e);
            if (e < least || v - lo > range) continue;       // (below lo: wraps to more)
            const int b = static_cast<int>((v - lo) >> shift);
            const uint64_t w = order == kByCount ? 1 : weight(list_value(e), c, s.pow);
            if (w != 0) add_wide(&s.sel_mass[b], w);
            atomicAdd(&s.sel_count[b], 1u);
        }
        __syncthreads();
        uint64_t m[8], own = 0;                              // every warp: 8 bins a lane, the largest values first
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint2 h = s.sel_mass[kSelectBins - 1 - lane * 8 - i];
            m[i] = (static_cast<uint64_t>(h.y) << 32) | h.x;
            own += m[i];
        }
        uint64_t before = warp_scan64(own, lane) - own;
        const uint32_t hit = __ballot_sync(0xffffffffu, before < limit && before + own >= limit);
        const int owner = hit != 0u ? __ffs(static_cast<int>(hit)) - 1 : 31;
        int bin = 0;
        bool open = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (open && before + m[i] >= limit) {
                bin = kSelectBins - 1 - lane * 8 - i;
                open = false;
            }
            if (open) before += m[i];
        }
        bin = __shfl_sync(0xffffffffu, bin, owner);
        limit -= __shfl_sync(0xffffffffu, before, owner);
        lo += static_cast<uint64_t>(bin) << shift;
        range = (1ull << shift) - 1;
        const bool one = s.sel_count[bin] == 1 || shift == 0;
        __syncthreads();
        if (one) break;
        if (tid < kSelectBins) {
            s.sel_mass[tid] = make_uint2(0u, 0u);
            s.sel_count[tid] = 0;
        }
        __syncthreads();
        shift = max(0, shift - 8);
    }
    for (int i = tid; i < n; i += NT) {
        const uint64_t e = s.list[i];
        if (e >= least && value(e) - lo <= range) s.sel_value = e;
    }
    __syncthreads();
    return s.sel_value;
}

// ---------------------------------------------------------------- kernel

template <typename E, int NT, bool kStaged>
__global__ void __launch_bounds__(NT, (kStaged ? 1024 : 2048) / NT) sample_tokens_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    SampleShared<NT>& s = *reinterpret_cast<SampleShared<NT>*>(smem);
    constexpr int kGroup = 16 / sizeof(E), kWarps = NT / 32, kEntries = kList / NT;
    constexpr bool kTable = NT == 1024;          // a CTA a row, no top-k: weights of bf16 values looked up
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.ctas;
    const int row = blockIdx.x / C;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    cluster_arrive();                            // every CTA runs before any writes into its shared memory
    ptx::griddep_wait();                         // a programmatic dependent: what came before is complete

    // ---- settings
    const float temperature = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.0f;
    const int k_in = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
    const float p_in = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.0f;
    const float m_in = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.0f;
    const float u = __ldg(a.u + row);
    const bool greedy = !(temperature > 0.0f);
    const bool use_k = !kTable && k_in > 0 && k_in < a.V, use_p = p_in < 1.0f, use_m = m_in > 0.0f;
    // Maxima that bound the k-th largest entry, 2048, or 1024 where they do for few threads (one row of 32000 9.0 -> 8.5 us): of
    // every thread, of two where the row has more threads, of parts of a thread's entries where it has fewer
    constexpr int kParts = kTable ? 1 : (kStaged ? (NT == 256 ? 4 : 1) : (sizeof(E) == 4 ? 2 : 4));
    const int up_to = NT == 256 && k_in <= kMaxima / 4 ? kMaxima / 2 : kMaxima;
    const int threads = C * NT, parts = threads >= up_to ? 1 : min(kParts, up_to / threads);
    const int num_maxima = min(up_to, threads * parts);
    const bool by_list = use_k && k_in <= kMaxTopK && (k_in <= num_maxima / 2 || a.V <= kList);

    // ---- the slice
    const E* logits = static_cast<const E*>(a.logits) + static_cast<int64_t>(row) * a.ld;
    constexpr int kDepth = kStaged ? 8 : (kTable ? 2 : 4);
    Slice<E, kStaged, kDepth> sl;
    sl.begin = min(a.V, static_cast<int>(rank) * a.slice);
    sl.end = min(a.V, sl.begin + a.slice);
    const int shift_in = static_cast<int>((reinterpret_cast<uintptr_t>(logits + sl.begin) & 15u) / sizeof(E));
    sl.first = sl.begin - shift_in;
    sl.data = reinterpret_cast<uint4*>(smem + sizeof(SampleShared<NT>));
    sl.row = logits;
    sl.most = largest<E>();
    sl.lane = lane;
    const int groups = sl.end > sl.begin ? (sl.end - sl.first + kGroup - 1) / kGroup : 0;
    const int per = (groups + kWarps - 1) / kWarps;
    sl.g0 = min(groups, warp * per);
    sl.g1 = min(groups, sl.g0 + per);
    // Numbers of the values of bf16 rows (below).  A CTA that has a row for itself counts as it reads; what has no bin of its
    // own it lists.
    uint32_t* counts = reinterpret_cast<uint32_t*>(&s);                      // over stage and list
    static_assert(offsetof(SampleShared<NT>, list) + sizeof(s.list) >= kValueBins * sizeof(uint32_t) + (kTable ? kOddList * sizeof(uint32_t) : 0), "counts");
    uint32_t* odd_list = counts + kValueBins;                                // indices
    auto count_values = [&](const uint4& r, int v, auto odd_one) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = (i & 1) != 0 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
            const uint32_t size = h & 0x7fffu, at = size - kFirstBits;
            if (at < static_cast<uint32_t>(kSide)) {
                const int d = static_cast<int>(at) + 1;
                atomicAdd(&counts[(h & 0x8000u) != 0u ? kSide - d : kSide + d], 1u);
            } else if (size < 0x7f80u) {                                     // (a row with +infinity does not go by counts)
                odd_one(h, v + i);
            }
        }
    };
    bool counting = false;
    if constexpr (kTable) counting = use_p && !use_k && !greedy;
    if (counting) {
        for (int i = tid; i < kValueBins; i += NT) counts[i] = 0;
        if (tid == 0) s.stage_count = 0;
        __syncthreads();
    }
    constexpr int kTracked = kStaged ? 1 : kParts;           // (a slice in shared memory is looked at again where parts are wanted)
    float top_part[kTracked];
    sl.take_in(top_part, [&](const uint4& r, int v) {
        if constexpr (kTable)
            if (counting)
                count_values(r, v, [&](uint32_t, int index) {
                    const uint32_t at = atomicAdd(&s.stage_count, 1u);
                    if (at < kOddList) odd_list[at] = static_cast<uint32_t>(index);
                });
    });
    float top_own = top_part[0];
#pragma unroll
    for (int i = 1; i < kTracked; ++i) top_own = fmaxf(top_own, top_part[i]);
    for (int i = tid; i < (1 << kPowBits) / 4; i += NT)
        reinterpret_cast<uint4*>(s.pow)[i] = __ldg(reinterpret_cast<const uint4*>(kPow.coarse) + i);
    if (tid == 0) {
        if (!counting) s.stage_count = 0;
        s.found = 0x7fffffff;
        const double r = 1024.0 * 1.4426950408889634074 / static_cast<double>(temperature);
        // (an infinite temperature: the smallest number, as 0 times the -infinity of masked entries, and of the places beside
        // the slice, would be NaN, whose bits say nothing of its size; weights of finite entries are 1 all the same)
        s.rh = r < FLT_MAX ? fmaxf(static_cast<float>(r), 0x1p-149f) : FLT_MAX;
        s.rl = r < FLT_MAX ? static_cast<float>(r - static_cast<double>(s.rh)) : 0.0f;
    }
    // by one thread: the fp64 unit is slow (by all of them 5 us).  At an infinite temperature all weights are 1, which no
    // min-p is above (infinity times the logarithm of 1 would be NaN)
    if (use_m && tid == 32)
        s.t_ln_min = temperature < INFINITY ? static_cast<double>(temperature) * log(static_cast<double>(fminf(m_in, 1.0f))) : -INFINITY;

    // ---- the largest entry
    cluster_wait();
    if (by_list && !greedy) {
        if (threads > up_to) {
            const float two = fmaxf(top_own, __shfl_xor_sync(0xffffffffu, top_own, 1));
            if ((tid & 1) == 0)
                for (int c = 0; c < C; ++c) put(&s.maxima[(rank * NT + tid) / 2], c, __float_as_uint(two));
        } else if (parts == 1) {
            for (int c = 0; c < C; ++c) put(&s.maxima[rank * NT + tid], c, __float_as_uint(top_own));
        } else {
            float top_of[kParts];
#pragma unroll
            for (int i = 0; i < kParts; ++i) top_of[i] = kStaged ? -INFINITY : top_part[i % kTracked];
            if constexpr (kStaged)
                sl.each_group([&](const uint4& r, int) {
                    float x[kGroup];
                    Slice<E, kStaged, kDepth>::unpack(r, x);
#pragma unroll
                    for (int e = 0; e < kGroup; ++e) top_of[e % kParts] = fmaxf(top_of[e % kParts], x[e]);
                });
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const float part = parts == kParts ? top_of[i] : fmaxf(top_of[i], top_of[(i + 2) % kParts]);
                for (int c = 0; c < C && i < parts; ++c) put(&s.maxima[(rank * parts + i) * NT + tid], c, __float_as_uint(part));
            }
        }
    }
    {
        const float m = warp_max(top_own);
        if (lane == 0) s.warp_max[warp] = m;
        __syncthreads();
        if (tid < C) {
            float t = -INFINITY;
            for (int w = 0; w < kWarps; ++w) t = fmaxf(t, s.warp_max[w]);
            put(&s.cta_max[rank], tid, __float_as_uint(t));
        }
    }
    cluster_sync();
    float top = -INFINITY;
    for (int c = 0; c < C; ++c) top = fmaxf(top, s.cta_max[c]);
    const Scale sc = make_scale(top, s.rh, s.rl);
    sl.most = top;

    float* probs = a.probs != nullptr ? a.probs + static_cast<int64_t>(row) * a.ld_probs : nullptr;
    auto clear_probs = [&]() {
        if (probs == nullptr) return;
        const bool vec = (reinterpret_cast<uintptr_t>(probs + sl.begin) & 15u) == 0;
        const int n = sl.end - sl.begin;
        if (vec) {
            for (int i = tid; i < n / 4; i += NT)
                __stcs(reinterpret_cast<float4*>(probs + sl.begin + 4 * i), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
            for (int i = n / 4 * 4 + tid; i < n; i += NT) probs[sl.begin + i] = 0.0f;
        } else {
            for (int i = tid; i < n; i += NT) probs[sl.begin + i] = 0.0f;
        }
    };

    if (greedy || sc.top == -INFINITY) {
        // ---- the first of the largest entries, or none
        clear_probs();
        if (sc.top > -INFINITY) {
            int v = 0x7fffffff;
            sl.each([&](float z, int i) {
                if (z == sc.top) v = min(v, i);
            });
            v = __reduce_min_sync(0xffffffffu, v);
            if (lane == 0 && v != 0x7fffffff) atomicMin(&s.found, v);
        }
        __syncthreads();
        if (tid == 0) put(&s.cta_index[rank], 0u, static_cast<uint32_t>(s.found));
        cluster_sync();                          // and the zeros come before the first CTA's 1
        if (rank == 0 && tid == 0) {
            int v = 0x7fffffff;
            for (int c = 0; c < C; ++c) v = min(v, s.cta_index[c]);
            if (v == 0x7fffffff) {
                raise_error(a.err, DSA_DEVERR_PROB);
                v = -1;
            } else if (probs != nullptr) {
                probs[v] = 1.0f;
            }
            a.tokens[row] = v;
        }
        return;
    }

    // Entries that `pick` takes, to the first CTA's list: their number (the same in every CTA), the list is whole if
    // that is at most kList and no CTA has more than its stage holds (else kList + 1 is returned).  Each CTA has a region
    // of the list; where one does not suffice they are sent again, packed.  The area of maxima, bins and stage is free.
    bool packed = false;
    // The entries are `floor` or more, and `pick` takes them; threads whose largest entry is below it have none (256 rows of
    // 131072 fp32 with probabilities, whose rows the L2 does not hold for a second read: 71 -> 64 us), other threads' groups
    // below it are passed over.
    auto collect = [&](float floor, auto pick) {
        __syncthreads();
        if (top_own >= floor) sl.each_group([&](const uint4& r, int v) {
            float x[kGroup];
            Slice<E, kStaged, kDepth>::unpack(r, x);
            float most = x[0];
#pragma unroll
            for (int i = 1; i < kGroup; ++i) most = fmaxf(most, x[i]);
            if (!(most >= floor) || most == -INFINITY) return;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const float z = kStaged ? x[i] : clean(x[i], sl.most);
                if (!(z >= floor) || z == -INFINITY || !pick(z, v + i)) continue;
                const uint32_t at = atomicAdd(&s.stage_count, 1u);
                const uint64_t e = list_entry(z, v + i);
                if (at < SampleShared<NT>::kStage) s.stage[at] = e;
                if (at < a.region) put(&s.list[rank * a.region + at], 0u, e);
            }
        });
        __syncthreads();
        const uint32_t n = s.stage_count;
        if (tid < C) put(&s.cta_count[rank], tid, n);
        cluster_sync();
        uint32_t all = 0, most = 0, before = 0;
        for (int c = 0; c < C; ++c) {
            const uint32_t m = s.cta_count[c];
            if (c < static_cast<int>(rank)) before += m;
            all += m;
            most = max(most, m);
        }
        packed = most > a.region;
        if (packed && all <= kList && most <= SampleShared<NT>::kStage) {
            for (uint32_t i = tid; i < n; i += NT) put(&s.list[before + i], 0u, s.stage[i]);
            cluster_sync();
        }
        return most <= max(a.region, static_cast<uint32_t>(SampleShared<NT>::kStage)) ? all : kList + 1u;
    };
    // Entry i of the list as it came in
    auto entry = [&](int i) {
        if (packed) return s.list[i];
        int c = 0;
        while (i >= static_cast<int>(s.cta_count[c])) i -= static_cast<int>(s.cta_count[c++]);
        return s.list[c * a.region + i];
    };
    // ... and the whole list without gaps
    auto pack = [&](int n) {
        if (packed) return;
        uint64_t v[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) v[e] = tid + e * NT < n ? entry(tid + e * NT) : 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEntries; ++e)
            if (tid + e * NT < n) s.list[tid + e * NT] = v[e];
        __syncthreads();
    };

    // smallest entry that min-p keeps
    float zmin = -INFINITY;
    if (use_m && tid == 0) {
        const double t = static_cast<double>(sc.top) + s.t_ln_min;
        zmin = static_cast<float>(t);
        if (static_cast<double>(zmin) < t) zmin = nextafterf(zmin, INFINITY);
        s.zmin = fminf(zmin, sc.top);
    }
    if (use_m) {
        __syncthreads();
        zmin = s.zmin;
    }
    // 1 / sum, by one thread as well
    auto inverse_of = [&](uint64_t sum) {
        if (tid == 0) {
            const double d = 1.0 / static_cast<double>(sum);
            const float hi = static_cast<float>(d);
            s.inv = make_float2(hi, static_cast<float>(d - static_cast<double>(hi)));
        }
        __syncthreads();
        return s.inv;
    };

    if constexpr (!kTable) if (by_list) {
        // ---- a bound that at least k entries reach: the k-th largest of the maxima, or a little less, by 256
        // bins of their range in turn
        constexpr int kKeys = kMaxima / NT;
        uint32_t key[kKeys];
        const uint32_t none = order_key(-INFINITY);
        uint32_t least = 0xffffffffu, finite = 0;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) {
            key[c] = c * NT + tid < num_maxima ? order_key(s.maxima[c * NT + tid]) : none;
            if (c * NT < num_maxima && key[c] != none) {
                least = min(least, key[c]);
                ++finite;
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        finite = __reduce_add_sync(0xffffffffu, finite);
        if (lane == 0) {
            s.warp_lo[warp] = least;
            s.warp_hi[warp] = finite;
        }
        if (tid < kSelectBins) s.sel_count[tid] = 0;
        __syncthreads();
        finite = 0;
        for (int i = 0; i < kWarps; ++i) {
            least = min(least, s.warp_lo[i]);
            finite += s.warp_hi[i];
        }
        const uint32_t wanted = static_cast<uint32_t>(k_in), enough = wanted + wanted / 8 + 8;
        float bound = -INFINITY;                             // fewer maxima than k: all entries
        if (finite >= wanted) {
            uint32_t lo = least, range = order_key(sc.top) - least, above = 0;
            int shift = max(0, 32 - __clz(static_cast<int>(range)) - 8);
            for (;;) {
#pragma unroll
                for (int c = 0; c < kKeys; ++c)
                    if (c * NT < num_maxima && key[c] != none && key[c] - lo <= range) atomicAdd(&s.sel_count[(key[c] - lo) >> shift], 1u);
                __syncthreads();
                uint32_t m[8], own = 0;                      // every warp: 8 bins a lane, the largest first
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m[i] = s.sel_count[kSelectBins - 1 - lane * 8 - i];
                    own += m[i];
                }
                uint32_t upto = own;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += o;
                }
                uint32_t at = above + upto - own;
                const int owner = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, at < wanted && at + own >= wanted))) - 1;
                int bin = 0;
                bool open = true;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (open && at + m[i] >= wanted) {
                        bin = kSelectBins - 1 - lane * 8 - i;
                        own = m[i];
                        open = false;
                    }
                    if (open) at += m[i];
                }
                bin = __shfl_sync(0xffffffffu, bin, owner);
                above = __shfl_sync(0xffffffffu, at, owner);
                own = __shfl_sync(0xffffffffu, own, owner);
                lo += static_cast<uint32_t>(bin) << shift;
                range = (1u << shift) - 1;
                if (above + own <= enough || shift == 0) break;
                __syncthreads();
                if (tid < kSelectBins) s.sel_count[tid] = 0;
                __syncthreads();
                shift = max(0, shift - 8);
            }
            bound = key_value(lo);
        }
        clear_probs();
        const uint32_t n_all = collect(bound, [](float, int) { return true; });
        if (n_all <= kList) {
            if (rank != 0) return;
            const int n = static_cast<int>(n_all), k = min(k_in, n);
            if (n <= kFew) {
                // ---- a few entries: each compares itself with all of them, twice
                uint64_t x = 0, w = 0;
                if (tid < n) {
                    x = entry(tid);
                    w = weight(list_value(x), sc, s.pow);
                    s.few.entry[tid] = x;
                    s.few.mass[tid] = w;
                }
                __syncthreads();
                int r = 0;
                uint64_t before = 0;
                if (tid < n) {
#pragma unroll 8
                    for (int j = 0; j < n; ++j)
                        if (s.few.entry[j] > x) {
                            ++r;
                            before += s.few.mass[j];
                        }
                    if (r == k - 1) s.limit = use_p ? max(scaled(p_in, before + w, true), uint64_t(1)) : ~0ull;
                }
                __syncthreads();
                const bool kept = tid < n && r < k && before < s.limit && list_value(x) >= zmin;
                const int nk = __syncthreads_count(kept);
                if (tid < n && !kept) s.few.mass[tid] = 0;
                if (kept && r == nk - 1) {                   // the last one kept: all before it are
                    s.sum = before + w;
                    s.limit = min(scaled(u, before + w, false), before + w - 1);
                }
                __syncthreads();
                const uint64_t target = s.limit;
                float2 inv{0.0f, 0.0f};
                if (probs != nullptr) inv = inverse_of(s.sum);
                if (kept) {
                    if (probs != nullptr) probs[list_index(x)] = probability(list_value(x), sc, s.pow, inv);
                    uint64_t upto = 0;                       // mass of the indices up to this one's
#pragma unroll 8
                    for (int j = 0; j < n; ++j) upto += static_cast<uint32_t>(s.few.entry[j]) >= static_cast<uint32_t>(x) ? s.few.mass[j] : 0;
                    if (upto > target && upto - w <= target) a.tokens[row] = list_index(x);
                }
                return;
            }
            // ---- more of them: three selections, by z for k, by z for p, by index for u
            pack(n);
            auto total = [&](uint64_t least, int slot) {
                uint64_t m = 0;
                for (int i = tid; i < n; i += NT)
                    if (s.list[i] >= least) m += weight(list_value(s.list[i]), sc, s.pow);
                return block_sum64(s, m, slot);
            };
            uint64_t least = n > k ? select(s, n, 0, kByCount, static_cast<uint64_t>(k), sc) : 0;
            if (use_p) {
                const uint64_t mass = total(least, 0);
                least = select(s, n, least, kByMass, max(scaled(p_in, mass, true), uint64_t(1)), sc);
            }
            least = max(least, static_cast<uint64_t>(order_key(zmin)) << 32);
            const uint64_t sum = total(least, 1);
            if (probs != nullptr) {
                const float2 inv = inverse_of(sum);
                for (int i = tid; i < n; i += NT)
                    if (s.list[i] >= least) probs[list_index(s.list[i])] = probability(list_value(s.list[i]), sc, s.pow, inv);
            }
            const uint64_t hit = select(s, n, least, kByIndex, min(scaled(u, sum, false), sum - 1) + 1, sc);
            if (tid == 0) a.tokens[row] = list_index(hit);
            return;
        }
    }

    int flip = 0;
    // Sum over the cluster; every thread of it gets it.
    auto cluster_sum = [&](uint64_t v) {
        const uint64_t t = block_sum64(s, v, flip);
        if (tid < C) put(&s.cta_sum[flip][rank], tid, t);
        cluster_sync();
        uint64_t all = 0;
        for (int c = 0; c < C; ++c) all += s.cta_sum[flip][c];
        flip ^= 1;
        return all;
    };
    // Narrows `cut` to the entries of it before which less than `limit` lies (their number, or their mass): the
    // smallest z above which less than the limit lies, by bisection, then the ties at it in the order of their indices.
    auto narrow = [&](const Cut& cut, bool masses, uint64_t limit) {
        uint32_t lo = order_key(-INFINITY), hi = order_key(sc.top);   // above lo: at least the limit (or lo is below all)
        uint64_t above = 0;
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            uint64_t n = 0;
            sl.each([&](float z, int v) {
                if (order_key(z) > mid && cut.keeps(z, v)) n += masses ? weight(z, sc, s.pow) : 1;
            });
            n = cluster_sum(n);
            if (n < limit) {
                hi = mid;
                above = n;
            } else {
                lo = mid;
            }
        }
        const float z_cut = key_value(hi);
        const uint64_t each = masses ? max(weight(z_cut, sc, s.pow), uint64_t(1)) : 1;
        const uint64_t ties = (limit - above + each - 1) / each;       // of those, in the order of their indices
        // the last of them
        uint64_t mine = 0;
        sl.each([&](float z, int v) { mine += z == z_cut && cut.keeps(z, v) ? 1 : 0; });
        const uint64_t in_warp = warp_sum64(mine);
        const int now = flip;
        const uint64_t all = cluster_sum(mine);
        uint64_t before = 0;
        for (int c = 0; c < static_cast<int>(rank); ++c) before += s.cta_sum[now][c];
        for (int w = 0; w < warp; ++w) before += s.warp_sum[now][w];
        Cut out{z_cut, cut.z == z_cut ? cut.index : 0x7fffffff};
        if (all > ties) {
            if (before < ties && before + in_warp >= ties) {
                for (int st = 0; st < sl.steps(); ++st) {
                    float x[kGroup];
                    const int v = sl.read(st, x);
                    uint32_t own = 0;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) own += x[i] == z_cut && cut.keeps(x[i], v + i) ? 1u : 0u;
                    uint64_t at = before + warp_scan64(own, lane) - own;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i)
                        if (x[i] == z_cut && cut.keeps(x[i], v + i) && ++at == ties)
                            for (int c = 0; c < C; ++c) put(&s.cut_index, c, static_cast<uint32_t>(v + i));
                    before += __reduce_add_sync(0xffffffffu, own);
                }
            }
            cluster_sync();
            out.index = s.cut_index;
            cluster_sync();                      // read by all before it is written again
        }
        return out;
    };

    Cut cut{-INFINITY, -1};
    bool counted = false;                        // the border is found, and the mass kept (sum of `mine`), without another pass
    bool by_counts = false;                      // ... from the numbers of values
    bool small = false;                          // the border lies among the numbers below 2^-9: `mine` is the mass above them
    uint64_t limit = 0;                          // of the mass that top-p keeps
    uint32_t kept_ties = 0;                      // of this CTA's entries at the border, where it lies among them
    uint64_t tie_weight = 0;
    uint64_t* table = reinterpret_cast<uint64_t*>(smem + sizeof(SampleShared<NT>));   // kTable: weights of the values that are kept
    uint64_t mine = 0;
    if constexpr (sizeof(E) == 2) {
        // ---- top-p alone, bf16: few distinct values, so their numbers say all.  A count is one addition in shared memory where a
        // mass is 30 operations and two of them; each weight is formed once a value, and once the border is known
        // the counts give the mass that a CTA keeps.  (300 rows of 100003: 258 -> 165 us)
        const int share = (kValueBins + C - 1) / C;                          // of the bins
        constexpr int kEach = kTable ? 5 : 3;                                // bins a thread
        if (use_p && !use_k && share <= kEach * NT && !sc.wide && sc.top < 128.0f && (!kTable || s.stage_count <= kOddList)) {
            static_assert(offsetof(SampleShared<NT>, list) + sizeof(s.list) >= kValueBins * sizeof(uint32_t), "counts");
            uint2* odd = s.sel_mass;                                         // masses of the numbers below 2^-9, and of those down from -2^7
            auto odd_one = [&](uint32_t h, int) {
                const uint64_t m = weight(__uint_as_float(h << 16), sc, s.pow);
                if (m != 0) add_wide(&odd[(h & 0x7fffu) < static_cast<uint32_t>(kFirstBits) ? 0 : 1], m);
            };
            __syncthreads();
            if (!kTable)
                for (int i = tid; i < kValueBins; i += NT) counts[i] = 0;
            if (tid < 2) odd[tid] = make_uint2(0u, 0u);
            __syncthreads();
            if constexpr (kTable) {
                for (int i = tid; i < static_cast<int>(s.stage_count); i += NT)
                    odd_one(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(logits)[odd_list[i]]), 0);
            } else {
                sl.each_group([&](const uint4& r, int v) { count_values(r, v, odd_one); });
            }
            cluster_sync();
            // this CTA's share of the bins, the largest values first, kEach a thread: masses over the cluster
            auto bin_at = [&](int i) {                                       // -1: none
                const int d = static_cast<int>(rank) * share + tid * kEach + i;
                return tid * kEach + i < share && d < kValueBins ? kValueBins - 1 - d : -1;
            };
            uint64_t own[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int bin = bin_at(i);
                own[i] = 0;
                if (bin >= 0) {
                    if (bin != kSide) {
                        uint32_t each[kMaxCtas], n = 0;
#pragma unroll
                        for (int c = 0; c < kMaxCtas; ++c) each[c] = kTable ? (c == 0 ? counts[bin] : 0) : (c < C ? get(&counts[bin], c) : 0);
#pragma unroll
                        for (int c = 0; c < kMaxCtas; ++c) n += each[c];
                        const uint64_t w = n == 0 ? 0 : weight(bin_value(bin), sc, s.pow);
                        if (kTable) table[bin] = w;
                        own[i] = n * w;
                    } else {
                        for (int c = 0; c < C; ++c) own[i] += wide(get2(&odd[0], c));
                    }
                }
                mine += own[i];
            }
            uint64_t rest = 0;                                               // behind all bins: what lies below -2^7
            if (static_cast<int>(rank) == C - 1 && tid == NT - 1)
                for (int c = 0; c < C; ++c) rest += wide(get2(&odd[1], c));
            const int now = flip;
            const uint64_t mass = cluster_sum(mine + rest);
            uint64_t before = 0;
            for (int c = 0; c < static_cast<int>(rank); ++c) before += s.cta_sum[now][c];
            for (int w = 0; w < warp; ++w) before += s.warp_sum[now][w];
            before += warp_scan64(mine + rest, lane) - (mine + rest);
            limit = max(scaled(p_in, mass, true), uint64_t(1));
            // the value of the border, and how many of the entries that are equal to it each CTA keeps (in all bins but the
            // two that hold several values)
            if (rest != 0 && before + mine < limit)
                for (int c = 0; c < C; ++c) put(&s.bin, c, 0xffffffffu);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (own[i] != 0 && before < limit && before + own[i] >= limit) {
                    const int bin = bin_at(i);
                    uint64_t left = 0;
                    if (bin != kSide) {
                        const uint64_t w = weight(bin_value(bin), sc, s.pow);
                        left = (limit - before + w - 1) / w;
                    }
                    uint32_t each[kMaxCtas];
#pragma unroll
                    for (int c = 0; c < kMaxCtas; ++c) each[c] = c < C ? get(&counts[bin], c) : 0;
#pragma unroll
                    for (int c = 0; c < kMaxCtas; ++c) {
                        const uint32_t q = static_cast<uint32_t>(min(static_cast<uint64_t>(each[c]), left));
                        left -= q;
                        if (c < C) {
                            put(&s.quota, c, q);
                            put(&s.bin, c, bin != kSide ? static_cast<uint32_t>(bin) : 0xfffffffeu);
                            put(&s.bin_before, c, before);
                        }
                    }
                }
                before += own[i];
            }
            cluster_sync();
            const int border = s.bin;
            const float z_cut = border >= 0 ? fmaxf(bin_value(border), zmin) : 0.0f;
            counted = by_counts = fabsf(z_cut) >= 0x1p-9f;                   // else below
            small = border == -2;
            if (small) {
                mine = 0;
                for (int b = kSide + 1 + tid; b < kValueBins; b += NT)
                    if (counts[b] != 0) mine += counts[b] * weight(bin_value(b), sc, s.pow);
                cluster_sync();                                              // the counts lie where the list does
            }
            if (counted) {
                cut = Cut{z_cut, 0x7fffffff};
                const uint32_t ties = counts[border], quota = s.quota;
                if (z_cut > bin_value(border)) {
                    // min-p keeps less: all that are not below it
                } else if (quota < ties) {
                    cut.index = -1;
                }
                kept_ties = z_cut > bin_value(border) || quota == ties ? 0 : quota;   // 0: all or none
                mine = 0;
                tie_weight = kept_ties > 0 ? weight(z_cut, sc, s.pow) : 0;
                for (int b = tid; b < kValueBins; b += NT) {
                    if (b == kSide) {
                        if (z_cut < 0.0f) mine += wide(odd[0]);
                        continue;
                    }
                    const float z = bin_value(b);
                    const uint32_t n = z > z_cut || (z == z_cut && cut.index == 0x7fffffff) ? counts[b] : (z == z_cut ? quota : 0);
                    if (n != 0) mine += n * (kTable ? table[b] : weight(z, sc, s.pow));
                }
                // no CTA reads the counts of another any more, and this one's lie where lists do
            }
        }
    }
    if constexpr (!kTable)
        if (use_k) cut = narrow(cut, false, static_cast<uint64_t>(k_in));
    if (use_p && !counted) {
        const float per_bin = sc.rh * (kBinsPerOctave / 1024.0f);
        auto place_of = [&](float z) { return fminf((sc.top - z) * per_bin, static_cast<float>(kBins - 1)); };
        __syncthreads();
        if (tid == 0) s.stage_count = 0;
        if (!small) {
            // ---- masses of bins of z, largest first
            for (int i = tid; i < kBins; i += NT) s.hist[i] = make_uint2(0u, 0u);
            __syncthreads();
            sl.each([&](float z, int v) {
                const uint64_t w = weight(z, sc, s.pow);
                if (w != 0 && cut.keeps(z, v)) add_wide(&s.hist[static_cast<int>(place_of(z))], w);
            });
            cluster_sync();
            // this CTA's share of the bins: sums over the cluster, then the mass of the share to every CTA
            const int share = kBins / C, b0 = static_cast<int>(rank) * share;      // C is a power of two
            uint64_t own[kBins / NT];
            mine = 0;
            const int each = (share + NT - 1) / NT;
#pragma unroll
            for (int i = 0; i < kBins / NT; ++i) {
                own[i] = 0;
                const int b = tid * each + i;
                if (i < each && b < share) {
                    uint2 h[kMaxCtas];
#pragma unroll
                    for (int c = 0; c < kMaxCtas; ++c) h[c] = c < C ? get2(&s.hist[b0 + b], c) : make_uint2(0u, 0u);
#pragma unroll
                    for (int c = 0; c < kMaxCtas; ++c) own[i] += wide(h[c]);
                }
                mine += own[i];
            }
            const int now = flip;
            const uint64_t mass = cluster_sum(mine);
            uint64_t before = 0;
            for (int c = 0; c < static_cast<int>(rank); ++c) before += s.cta_sum[now][c];
            for (int w = 0; w < warp; ++w) before += s.warp_sum[now][w];
            before += warp_scan64(mine, lane) - mine;
            limit = max(scaled(p_in, mass, true), uint64_t(1));
            // the bin of the last entry before which less than the limit lies: mass up to it reaches the limit
#pragma unroll
            for (int i = 0; i < kBins / NT; ++i) {
                if (own[i] != 0 && before < limit && before + own[i] >= limit)
                    for (int c = 0; c < C; ++c) {
                        put(&s.bin, c, static_cast<uint32_t>(b0 + tid * each + i));
                        put(&s.bin_before, c, before);
                    }
                before += own[i];
            }
            cluster_sync();
            mine = 0;                                                      // this CTA's mass above the border's bin
            if constexpr (!kTable)
                for (int b = tid; b < s.bin; b += NT) mine += wide(s.hist[b]);
        }
        const float bin = static_cast<float>(s.bin);
        const uint64_t bin_before = s.bin_before;
        const uint32_t n = collect(small ? -0x1p-9f : -INFINITY, [&](float z, int v) {
            if (small) return fabsf(z) < 0x1p-9f;
            const float b = place_of(z);
            return b >= bin && b < bin + 1.0f && cut.keeps(z, v);
        });
        if (n <= kList) {
            if (rank == 0) {
                pack(static_cast<int>(n));
                const uint64_t last = select(s, static_cast<int>(n), 0, kByMass, limit - bin_before, sc);
                // and each CTA's mass in the bin
                if (tid < kMaxCtas) s.sel_mass[tid] = make_uint2(0u, 0u);
                __syncthreads();
                for (int i = tid; (!kTable || small) && i < static_cast<int>(n); i += NT)
                    if (s.list[i] >= last) add_wide(&s.sel_mass[list_index(s.list[i]) / a.slice], weight(list_value(s.list[i]), sc, s.pow));
                __syncthreads();
                if (tid < C) {
                    put(&s.border_mass, tid, wide(s.sel_mass[tid]));
                    put(&s.cut_key, tid, static_cast<uint32_t>(last >> 32));
                    put(&s.cut_index, tid, static_cast<uint32_t>(list_index(last)));
                }
            }
            cluster_sync();
            cut = Cut{key_value(s.cut_key), s.cut_index};
            counted = (!kTable || small) && !(zmin > cut.z);
            if (tid == 0) mine += s.border_mass;
        } else {
            cut = narrow(cut, true, limit);
        }
    }
    if (zmin > cut.z) cut = Cut{zmin, 0x7fffffff};

    // ---- the sum of what is kept, by warps; the warp with the border looks again
    auto sum_up = [&]() {
        mine = 0;
        sl.each([&](float z, int v) {
            if (cut.keeps(z, v)) mine += weight(z, sc, s.pow);
        });
    };
    if (!counted) sum_up();
    int now = flip;
    __syncthreads();
    const uint64_t sum = cluster_sum(mine);
    const uint64_t target = min(scaled(u, sum, false), sum - 1);       // u of 1 or more: the last one kept
    uint64_t before = 0;
    for (int c = 0; c < static_cast<int>(rank); ++c) before += s.cta_sum[now][c];
    bool drawn = false;
    if constexpr (kTable) {
        if (by_counts) {
            // ---- the draw, every entry's weight from the table; entries equal to the border's value are counted, the first
            // kept_ties of them, in the order of the indices, are kept
            const uint32_t border_bits = kept_ties > 0 ? __float_as_uint(cut.z) >> 16 : 0xffffu;      // (no number)
            const float below = kept_ties == 0 ? nextafterf(cut.z, -INFINITY) : cut.z;               // kept: z > below
            auto bin_weight = [&](uint32_t h) -> uint64_t {
                const uint32_t at = (h & 0x7fffu) - kFirstBits;
                const int neg = static_cast<int>(h << 16) >> 31, d = (static_cast<int>(at + 1) ^ neg) - neg;
                return __uint_as_float(h << 16) > below && at < static_cast<uint32_t>(kSide) ? table[kSide + d] : 0;
            };
            // an entry without a bin of its own
            auto odd_weight = [&](uint32_t h) -> uint64_t {
                const float z = __uint_as_float(h << 16);
                return z > below && (h & 0x7fffu) < static_cast<uint32_t>(kFirstBits) ? weight(z, sc, s.pow) : 0;
            };
            auto half = [](const uint4& r, int i) {
                const uint32_t w = (i >> 1) == 0 ? r.x : ((i >> 1) == 1 ? r.y : ((i >> 1) == 2 ? r.z : r.w));
                return (i & 1) != 0 ? w >> 16 : w & 0xffffu;
            };
            uint64_t own = 0;
            uint32_t ties = 0;
            __syncthreads();                                           // the table is written
            sl.each_group([&](const uint4& r, int) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    own += bin_weight(half(r, i));
                    ties += half(r, i) == border_bits ? 1u : 0u;
                }
            });
            own = warp_sum64(own);
            ties = __reduce_add_sync(0xffffffffu, ties);
            uint2* odd_sums = s.sel_mass;                              // of each warp's entries without a bin
            if (lane == 0) {
                s.warp_sum[flip][warp] = own;
                s.warp_lo[warp] = ties;
            }
            if (tid < kWarps) odd_sums[tid] = make_uint2(0u, 0u);
            __syncthreads();
            if (below < 0.0f)
                for (int i = tid; i < static_cast<int>(s.stage_count); i += NT) {
                    const int v = static_cast<int>(odd_list[i]);
                    const uint64_t w = odd_weight(reinterpret_cast<const uint16_t*>(logits)[v]);
                    if (w != 0) add_wide(&odd_sums[(v - sl.first) / kGroup / per], w);
                }
            __syncthreads();
            // lane l: warp l's
            auto scan32 = [&](uint32_t v) {
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += o;
                }
                return v;
            };
            const uint32_t t_own = s.warp_lo[lane], t_before = scan32(t_own) - t_own;
            const uint32_t t_kept = min(t_own, kept_ties - min(kept_ties, t_before));
            const uint64_t m_own = s.warp_sum[flip][lane] + wide(odd_sums[lane]) + t_kept * tie_weight, m_upto = warp_scan64(m_own, lane);
            uint64_t upto = __shfl_sync(0xffffffffu, m_upto, warp);
            uint64_t from = upto - __shfl_sync(0xffffffffu, m_own, warp);
            uint32_t seen = __shfl_sync(0xffffffffu, t_before, warp);
            if (from <= target && target < upto) {
                bool done = false;
                constexpr int kLoads = 4;                              // steps' groups loaded together
                uint4 next[kLoads];
                for (int st = 0; st < sl.steps() && !done; ++st) {
                    if (st % kLoads == 0) {
#pragma unroll
                        for (int j = 0; j < kLoads; ++j) {
                            const int g = sl.g0 + (st + j) * 32 + lane;
                            next[j] = g < sl.g1 ? sl.raw(g) : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
                        }
                    }
                    const int g = sl.g0 + st * 32 + lane;
                    const uint4 r = next[0];
#pragma unroll
                    for (int j = 1; j < kLoads; ++j) next[j - 1] = next[j];
                    uint32_t n = 0;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) n += half(r, i) == border_bits ? 1u : 0u;
                    uint32_t tie = seen + scan32(n) - n;               // ties in front of this lane's
                    seen = __shfl_sync(0xffffffffu, tie + n, 31);
                    uint64_t w[kGroup], sum_own = 0;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) {
                        const bool is_tie = half(r, i) == border_bits;
                        w[i] = is_tie ? (tie < kept_ties ? tie_weight : 0) : bin_weight(half(r, i)) + odd_weight(half(r, i));
                        tie += is_tie ? 1u : 0u;
                        sum_own += w[i];
                    }
                    const uint64_t inc = from + warp_scan64(sum_own, lane);
                    uint64_t at = inc - sum_own;
                    if (at <= target && target < inc) {
                        int token = -1;
#pragma unroll
                        for (int i = 0; i < kGroup; ++i) {
                            at += w[i];
                            if (token < 0 && at > target) token = sl.group_index(g) + i;
                        }
                        a.tokens[row] = token;
                        done = true;
                    }
                    done = __any_sync(0xffffffffu, done);
                    from = __shfl_sync(0xffffffffu, inc, 31);
                }
            }
            if (probs == nullptr) return;
            drawn = true;
            __syncthreads();
        }
    }
    if (counted) {                                                     // only the CTA with the border needs its warps' sums
        const bool here = !drawn && before <= target && target < before + s.cta_sum[now][rank];
        if (kept_ties > 0 && (here || probs != nullptr)) {             // the last one kept, in the order of the indices
            uint64_t n = 0;
            sl.each([&](float z, int) { n += z == cut.z ? 1 : 0; });
            const uint64_t in_warp = warp_sum64(n);
            block_sum64(s, n, flip);
            uint64_t seen = 0;
            for (int w = 0; w < warp; ++w) seen += s.warp_sum[flip][w];
            if (seen < kept_ties && seen + in_warp >= kept_ties) {
                for (int st = 0; st < sl.steps(); ++st) {
                    float x[kGroup];
                    const int v = sl.read(st, x);
                    uint32_t own = 0;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i) own += x[i] == cut.z ? 1u : 0u;
                    uint64_t at = seen + warp_scan64(own, lane) - own;
#pragma unroll
                    for (int i = 0; i < kGroup; ++i)
                        if (x[i] == cut.z && ++at == kept_ties) s.cut_index = v + i;
                    seen += __reduce_add_sync(0xffffffffu, own);
                }
            }
            __syncthreads();
            cut.index = s.cut_index;
        }
        if (here) {
            sum_up();
            now = flip;
            __syncthreads();
            block_sum64(s, mine, now);
        } else {
            mine = 0;
        }
    }
    const uint64_t in_warp = warp_sum64(mine);
    for (int w = 0; w < warp; ++w) before += s.warp_sum[now][w];
    if (before <= target && target < before + in_warp) {
        bool done = false;
        for (int st = 0; st < sl.steps() && !done; ++st) {
            float x[kGroup];
            const int v = sl.read(st, x);
            uint64_t w[kGroup], own = 0;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                w[i] = cut.keeps(x[i], v + i) ? weight(x[i], sc, s.pow) : 0;
                own += w[i];
            }
            const uint64_t inc = before + warp_scan64(own, lane);
            uint64_t at = inc - own;
            if (at <= target && target < inc) {
                int token = -1;
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    at += w[i];
                    if (token < 0 && at > target) token = v + i;
                }
                a.tokens[row] = token;
                done = true;
            }
            done = __any_sync(0xffffffffu, done);
            before = __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    if (probs != nullptr) {
        const float2 inv = inverse_of(sum);
        for (int g = sl.g0 + lane; g < sl.g1; g += 32) {
            float x[kGroup];
            sl.values(sl.raw(g), x);
            const int v = sl.group_index(g);
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                if (v + i >= sl.begin && v + i < sl.end)
                    probs[v + i] = cut.keeps(x[i], v + i) ? probability(x[i], sc, s.pow, inv) : 0.0f;
        }
    }
    // (nothing reaches into another CTA's shared memory after the barrier of the sum)
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_sample_tokens(const void* logits, int64_t ld, int32_t V, int32_t R, uint32_t flags,
                                        const float* temperature, const int32_t* top_k, const float* top_p,
                                        const float* min_p, const float* u, int32_t* tokens, float* probs,
                                        int64_t ld_probs, int32_t* dev_err, void* stream) {
    using namespace dsa;
    if ((flags & ~DSA_LOGITS_BF16) != 0u) return DSA_ERR_INVALID_ARG;
    const bool bf16 = (flags & DSA_LOGITS_BF16) != 0u;
    if (R < 0 || V < 1) return DSA_ERR_INVALID_ARG;
    if (V > kMaxSampleVocab || R > 0x7fffffff / kMaxCtas) return DSA_ERR_UNSUPPORTED;
    if (R == 0) return DSA_OK;
    if (!logits || !u || !tokens || ld < V || (probs != nullptr && ld_probs < V)) return DSA_ERR_INVALID_ARG;
    const uintptr_t align = bf16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % align != 0 || reinterpret_cast<uintptr_t>(probs) % 4 != 0) return DSA_ERR_INVALID_ARG;
    // the outputs may not lie over the inputs or each other: a CTA writes its own while others still read (its row's settings
    // too, which are loaded where they are used)
    const size_t n_logits = (static_cast<size_t>(R - 1) * ld + V) * align, n_probs = (static_cast<size_t>(R - 1) * ld_probs + V) * 4;
    const size_t n_row = static_cast<size_t>(R) * 4;
    if (overlap(probs, n_probs, logits, n_logits) || overlap(tokens, n_row, logits, n_logits) || overlap(tokens, n_row, probs, n_probs))
        return DSA_ERR_INVALID_ARG;
    for (const void* in : {static_cast<const void*>(temperature), static_cast<const void*>(top_k), static_cast<const void*>(top_p),
                           static_cast<const void*>(min_p), static_cast<const void*>(u)})
        if (overlap(probs, n_probs, in, n_row) || overlap(tokens, n_row, in, n_row)) return DSA_ERR_INVALID_ARG;
    int ctas = 1;
    while (ctas < kMaxCtas && V > ctas * 2048) ctas *= 2;
    // many rows: not more CTAs than need be (a top-k of up to 1024 wants four), with 8192 entries or so each (k = 50: 512 rows of
    // 16000 93 -> 51 us, 160 of 32000 31 -> 19; top-p alone: 512 of 16000 174 -> 121, but 120 of 32000 64 -> 77)
    const int64_t enough = (top_k != nullptr ? 4 : 8) * static_cast<int64_t>(device_sm_count());
    if (ctas == 8 && R * static_cast<int64_t>(ctas) > enough && V <= 8 * 8192) ctas = 4;
    // Staged unless most of the work is rows with a top-k, and there are enough of them to fill the GPU several
    // times: then more CTAs an SM count for more (256 rows of 131072 with k = 50 and probabilities 134 -> 100 us; 64 rows of
    // mixed settings 53 -> 63, 300 with top-p alone 268 -> 361)
    const int64_t slots = 4 * static_cast<int64_t>(device_sm_count());
    const bool staged = top_k == nullptr || R * static_cast<int64_t>(ctas) <= slots;
    if (!staged) {
        // A CTA takes about as long as 16384 entries for what it does besides reading: as many CTAs a row as make the least of
        // that times the waves.  Not more than 32768 entries for one: rows without a top-k go over them several times (300 rows
        // of 131072 bf16, k = 50: four CTAs a row 43 us, two 34, but with a setting each 111 and 203).  Not one for fp32, where
        // a thread keeps two maxima (registers).  With this rule instead of eight CTAs a row: 300 rows of 131072 bf16 65 -> 43
        // us, with a setting each 131 -> 111, 300 of 32000 33 -> 21, 512 of 16000 54 -> 23, with a setting each 112 -> 84
        int64_t best = INT64_MAX;
        const int most = ctas;
        for (int c = most; c >= std::min(most, bf16 ? 1 : 2); c /= 2) {
            const int64_t part = (V + c - 1) / c, time = (R * static_cast<int64_t>(c) + slots - 1) / slots * (16384 + part);
            if (c < most && part > 32768) break;
            if (time < best) {
                best = time;
                ctas = c;
            }
        }
    }
    const int slice = ((V + ctas - 1) / ctas + 7) / 8 * 8;
    const size_t bytes = (static_cast<size_t>(slice) * align + 15) / 16 * 16 + 16;
    const bool large = bytes > 40 * 1024 || !staged;
    size_t smem = (staged ? bytes : 0) + (large ? sizeof(SampleShared<512>) : sizeof(SampleShared<256>));
    SampleArgs a{logits, ld, V, temperature, top_k, top_p, min_p, u, tokens, probs, ld_probs, ctas, slice, static_cast<uint32_t>(kList / ctas), dev_err};
    using Kernel = void (*)(SampleArgs);
    // A CTA a row where top-p alone goes by counts of values and there are rows enough: no exchanges between CTAs, and what
    // each CTA does for all values is done once a row (rows x entries: 300 x 100003 135 -> 88 us, 512 x 16000 162 -> 65,
    // 80 x 100000 72 -> 59; 40 x 100000 46 -> 59, 512 x 1000 34 -> 54)
    const bool single = bf16 && top_k == nullptr && top_p != nullptr && R >= kSingleRows && V > kSingleVocab;
    static const Kernel kernels[2][3] = {
        {sample_tokens_kernel<float, 512, false>, sample_tokens_kernel<float, 256, true>, sample_tokens_kernel<float, 512, true>},
        {sample_tokens_kernel<uint16_t, 512, false>, sample_tokens_kernel<uint16_t, 256, true>, sample_tokens_kernel<uint16_t, 512, true>}};
    const void* kernel = reinterpret_cast<const void*>(kernels[bf16 ? 1 : 0][!staged ? 0 : (large ? 2 : 1)]);
    int threads = large ? 512 : 256;
    if (single) {
        kernel = reinterpret_cast<const void*>(&sample_tokens_kernel<uint16_t, 1024, false>);
        threads = 1024;
        ctas = a.ctas = 1;
        a.slice = (V + 7) / 8 * 8;
        a.region = kList;
        smem = sizeof(SampleShared<1024>) + kValueBins * sizeof(uint64_t);
    }
    // (the same limit in every call: another thread's may come between this and the launch)
    if (smem > kMaxSmem || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
        return DSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(R) * ctas);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[] = {&a};
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}
