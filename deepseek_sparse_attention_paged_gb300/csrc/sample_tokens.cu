// sample_tokens.cu -- the next token of every row of logits: temperature, top-k, top-p and min-p, then a draw
// with a given random number (sm_103a).
//
// Mathematics: w = 2^((z - max z) log2 e / temperature); order: larger z first, ties by index.  top-k keeps the
// first k; top-p those of them before which less than p of their mass lies; min-p those with w >= min_p.  The
// token is the least v with sum_{i <= v} w_i > u sum w over what is kept.
//
// Sums: a token must not depend on how a sum is split, and a border between two of 10^5 tokens is missed where
// sums are off by 10^-5 of a weight.  So a weight is formed to about 2^-35 of itself (z - max z and its product
// with log2 e / t as unevaluated pairs of fp32, 2^(j / 1024) from a table of 46-bit integers, the rest a cubic)
// and held as an integer, 2^45 the largest: integer sums do not round, in any order, and u S and p M are compared
// exactly (24 x 64 bits).  The fp64 unit would take ten times as long as the read of the row.
//
// A row is split over the CTAs of a cluster, each with a slice of it in shared memory: logits are read from global
// memory once.
//   * top-k up to 1024: the k-th largest of all threads' maxima is a bound from below that few more than k
//     entries pass (with G threads about -G ln(1 - k / G)); those go to the first CTA, which sorts them and does the
//     rest alone.
//   * top-p without top-k: masses of 1024 bins of z (32 an octave of w) find the bin of the border; its entries
//     go to the first CTA, which sorts them and finds the last one kept.  A second pass sums what is kept.
//   * where more entries than fit (2048) come together (ties, a temperature far above 1), or for a larger top-k:
//     bisection over the 32 bits of z, a pass over the slices each.
#include <float.h>

#include <algorithm>

#include "dsa_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kList = 2048;                    // entries that the first CTA sorts
constexpr int kMaxTopK = 1024;
constexpr int kBins = 1024, kBinsPerOctave = 32;
constexpr int kOne = 45;                       // fraction bits of a weight
constexpr int kMaxSampleVocab = 1 << 18;       // sums of weights stay below 2^63
constexpr int kPowBits = 10;

// 2^(j / 1024) with kOne fraction bits, by the exponential series in 62-bit fixed point.
struct PowTable {
    uint64_t v[1 << kPowBits];
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
        t.v[j] = static_cast<uint64_t>((sum + (u128(1) << (61 - kOne))) >> (62 - kOne));
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
    int32_t* err;
};

struct alignas(16) SampleShared {
    union {
        float maxima[kMaxCtas * kThreads];     // every thread's largest entry, of all CTAs
        uint2 hist[kBins];                     // masses (low and high word)
        uint64_t stage[kList];                 // entries of this CTA on their way to the first one
    };
    uint64_t list[kList];                      // first CTA: (order key of z, ~index)
    uint64_t pow[1 << kPowBits];
    // written by all CTAs of the cluster
    float cta_max[kMaxCtas];
    int cta_index[kMaxCtas];
    uint32_t cta_count[kMaxCtas];
    uint64_t cta_sum[2][kMaxCtas];
    uint32_t list_count;
    uint32_t cut_key;
    int cut_index;
    int bin;
    uint64_t bin_before;
    // this CTA's
    uint64_t warp_sum[2][kWarps];
    float warp_max[kWarps];
    uint32_t stage_count, stage_base;
    int found;
    float rh, rl, zmin;
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
__device__ __forceinline__ uint2 get2(const void* p, uint32_t rank) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t add_remote(void* p, uint32_t rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote(p, rank)), "r"(v) : "memory");
    return old;
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

// max z, log2 e / t = rh + rl
struct Scale {
    float top, rh, rl;
};

// log2 w, as a pair
__device__ __forceinline__ float log2_weight(float z, const Scale& c, float& lo) {
    const float s = __fsub_rn(z, c.top);
    const float e = two_sum_err(z, -c.top, s);
    const float y = __fmul_rn(s, c.rh);
    lo = __fadd_rn(__fmaf_rn(s, c.rh, -y), __fmaf_rn(s, c.rl, __fmul_rn(e, c.rh)));
    return y;
}
// w 2^kOne = x 2^-shift, x of 46 bits, for y = log2 w in [-200, 0]
__device__ __forceinline__ uint64_t power(float y, float lo, const uint64_t* pow, int& shift) {
    constexpr float kMagic = 12582912.0f;                    // 1.5 2^23: adding it rounds to whole numbers
    const float t = __fmaf_rn(y, 1024.0f, kMagic);
    const int n = __float_as_int(t) - __float_as_int(kMagic);
    const float f = __fadd_rn(__fmaf_rn(__fsub_rn(t, kMagic), -1.0f / 1024.0f, y), lo);   // |f| <= 2^-11
    // 2^f - 1 with 41 fraction bits: ln 2, ln^2 2 / 2, ln^3 2 / 6 times 2^41
    constexpr float c1 = 0.69314718055994531f * 0x1p41f, c2 = 0.24022650695910072f * 0x1p41f, c3 = 0.05550410866482158f * 0x1p41f;
    const int g = __float2int_rn(f * __fmaf_rn(f, __fmaf_rn(f, c3, c2), c1));
    const uint64_t p = pow[n & ((1 << kPowBits) - 1)];
    shift = -(n >> kPowBits);
    return p + static_cast<uint64_t>((static_cast<int64_t>(static_cast<int>(p >> 15)) * g) >> 26);
}
// w 2^kOne as a whole number; 0 below 2^-46
__device__ __forceinline__ uint64_t weight(float z, const Scale& c, const uint64_t* pow) {
    float lo;
    const float y = log2_weight(z, c, lo);
    if (!(y > -46.0f)) return 0;
    int shift;
    const uint64_t x = power(y, lo, pow, shift);
    return (x + ((1ull << shift) >> 1)) >> shift;
}

// 1 / sum as a pair; probabilities from it
struct Inverse {
    float hi, lo;
};
__device__ __forceinline__ Inverse inverse(uint64_t sum) {
    const double d = 1.0 / static_cast<double>(sum);
    const float hi = static_cast<float>(d);
    return Inverse{hi, static_cast<float>(d - static_cast<double>(hi))};
}
__device__ __forceinline__ float probability(float z, const Scale& c, const uint64_t* pow, Inverse inv) {
    float lo;
    const float y = log2_weight(z, c, lo);
    if (!(y > -160.0f)) return 0.0f;
    int shift;
    const uint64_t x = power(y, lo, pow, shift);
    const float xh = static_cast<float>(static_cast<uint32_t>(x >> 22)), xl = static_cast<float>(static_cast<uint32_t>(x) & 0x3fffffu) * 0x1p-22f;
    const float p = __fmaf_rn(xh, inv.hi, __fmaf_rn(xh, inv.lo, xl * inv.hi));
    const int first = min(shift, 100);                       // a subnormal number rounds once
    return p * __int_as_float((127 + 22 - first) << 23) * __int_as_float((127 - (shift - first)) << 23);
}

// floor(a s), rounded up where `up` is set and it is not whole: a >= 0 finite, s < 2^63; saturates
__device__ __forceinline__ uint64_t scaled(float a, uint64_t s, bool up) {
    if (!(a > 0.0f)) return 0;
    const uint32_t b = __float_as_uint(a);
    const int ex = static_cast<int>(b >> 23);
    const uint64_t m = ex != 0 ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int right = 150 - max(ex, 1);                      // a = m 2^-right
    uint64_t lo = m * s, hi = __umul64hi(m, s);
    if (right <= 0) return ~0ull >> 1;                       // a >= 2^23
    uint64_t out, rest;
    if (right < 64) {
        if ((hi >> right) != 0u) return ~0ull >> 1;
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

// A CTA's slice in shared memory: groups of 16 bytes that lie as they do in global memory (on 16-byte
// boundaries), entries outside the slice -infinity.  Warp w has the groups [w per, (w + 1) per), its lanes
// one after the other: a thread reads only what it wrote itself, and warps, steps and lanes follow the indices.
template <typename E>
struct Slice {
    static constexpr int kGroup = 16 / sizeof(E);
    uint4* data;
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
    // entries of this lane's group of a step; -infinity past the warp's groups
    __device__ __forceinline__ int read(int step, float (&x)[kGroup]) const {
        const int g = g0 + step * 32 + lane;
        if (g < g1) {
            unpack(data[g], x);
        } else {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) x[i] = -INFINITY;
        }
        return group_index(g);
    }
    // f(z, index) for every entry of this thread
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        for (int g = g0 + lane; g < g1; g += 32) {
            float x[kGroup];
            unpack(data[g], x);
            const int v = group_index(g);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) f(x[i], v + i);
        }
    }
};

// From global memory: NaN counts as -infinity, +infinity as the largest number of the type.
template <typename E>
__device__ __forceinline__ uint32_t clean(uint32_t w) {
    if constexpr (sizeof(E) == 4) {
        return __float_as_uint(fminf(fmaxf(__uint_as_float(w), -INFINITY), FLT_MAX));
    } else {
        const float lo = fminf(fmaxf(bf16_lo(w), -INFINITY), __uint_as_float(0x7f7f0000u));
        const float hi = fminf(fmaxf(bf16_hi(w), -INFINITY), __uint_as_float(0x7f7f0000u));
        return (__float_as_uint(lo) >> 16) | __float_as_uint(hi);
    }
}

template <typename E>
__device__ __forceinline__ uint4 load_group(const E* row, int v, int begin, int end) {
    constexpr int n = 16 / sizeof(E);
    uint32_t w[4];
    if (v >= begin && v + n <= end) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(row + v));
        w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
    } else if constexpr (sizeof(E) == 4) {
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
    return make_uint4(clean<E>(w[0]), clean<E>(w[1]), clean<E>(w[2]), clean<E>(w[3]));
}

// ---------------------------------------------------------------- the first CTA's list

// Largest first.  Few entries: each counts those before it.
__device__ void sort_list(uint64_t* a, int n) {
    const int tid = threadIdx.x;
    if (n <= 256) {
        const uint64_t x = tid < n ? a[tid] : 0;
        int r = 0;
        if (tid < n)
            for (int j = 0; j < n; ++j) r += a[j] > x ? 1 : 0;
        __syncthreads();
        if (tid < n) a[r] = x;
        __syncthreads();
        return;
    }
    int p = 512;
    while (p < n) p <<= 1;
    for (int i = n + tid; i < p; i += kThreads) a[i] = 0;    // below every entry
    __syncthreads();
    for (int k = 2; k <= p; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = tid; i < p; i += kThreads) {
                const int o = i ^ j;
                if (o > i) {
                    const uint64_t x = a[i], y = a[o];
                    if ((x < y) == ((i & k) == 0)) {
                        a[i] = y;
                        a[o] = x;
                    }
                }
            }
            __syncthreads();
        }
}

__device__ __forceinline__ float list_value(uint64_t e) { return key_value(static_cast<uint32_t>(e >> 32)); }
__device__ __forceinline__ int list_index(uint64_t e) { return static_cast<int>(~static_cast<uint32_t>(e)); }

// Sum over the block; all threads get it.  `slot` alternates between two calls in a row.
__device__ __forceinline__ uint64_t block_sum64(SampleShared& s, uint64_t v, int slot) {
    v = warp_sum64(v);
    if ((threadIdx.x & 31) == 0) s.warp_sum[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s.warp_sum[slot][w];
    return t;
}

constexpr int kPerThread = kList / kThreads;

// Weights of the sorted entries list[0, n): thread t has entries t kPerThread ..; `before` the mass in front of each.
__device__ __forceinline__ uint64_t list_masses(SampleShared& s, int n, const Scale& c, uint64_t (&w)[kPerThread],
                                                uint64_t (&before)[kPerThread]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t own = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int at = threadIdx.x * kPerThread + i;
        w[i] = at < n ? weight(list_value(s.list[at]), c, s.pow) : 0;
        before[i] = own;
        own += w[i];
    }
    const uint64_t inc = warp_scan64(own, lane);
    __syncthreads();                                         // warp_sum is free
    if (lane == 31) s.warp_sum[0][warp] = inc;
    __syncthreads();
    uint64_t base = inc - own, total = 0;
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) base += s.warp_sum[0][i];
        total += s.warp_sum[0][i];
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) before[i] += base;
    return total;
}

// ---------------------------------------------------------------- kernel

template <typename E>
__global__ void __launch_bounds__(kThreads) sample_tokens_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
    constexpr int kGroup = 16 / sizeof(E);
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
    const bool use_k = k_in > 0 && k_in < a.V, use_p = p_in < 1.0f, use_m = m_in > 0.0f;
    const bool by_list = use_k && k_in <= min(kMaxTopK, C * kThreads / 2);

    // ---- the slice
    const E* logits = static_cast<const E*>(a.logits) + static_cast<int64_t>(row) * a.ld;
    Slice<E> sl;
    sl.begin = min(a.V, static_cast<int>(rank) * a.slice);
    sl.end = min(a.V, sl.begin + a.slice);
    const int shift_in = static_cast<int>((reinterpret_cast<uintptr_t>(logits + sl.begin) & 15u) / sizeof(E));
    sl.first = sl.begin - shift_in;
    sl.data = reinterpret_cast<uint4*>(smem + sizeof(SampleShared));
    sl.lane = lane;
    const int groups = sl.end > sl.begin ? (sl.end - sl.first + kGroup - 1) / kGroup : 0;
    const int per = (groups + kWarps - 1) / kWarps;
    sl.g0 = min(groups, warp * per);
    sl.g1 = min(groups, sl.g0 + per);
    float top_own = -INFINITY;
    for (int g = sl.g0 + lane; g < sl.g1; g += 32 * 8) {
        uint4 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (g + 32 * i < sl.g1) r[i] = load_group<E>(logits, sl.group_index(g + 32 * i), sl.begin, sl.end);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (g + 32 * i < sl.g1) {
                sl.data[g + 32 * i] = r[i];
                float x[kGroup];
                Slice<E>::unpack(r[i], x);
#pragma unroll
                for (int e = 0; e < kGroup; ++e) top_own = fmaxf(top_own, x[e]);
            }
    }
    for (int i = tid; i < (1 << kPowBits); i += kThreads) s.pow[i] = kPow.v[i];
    if (tid == 0) {
        s.list_count = 0;
        s.stage_count = 0;
        s.found = 0x7fffffff;
        const double r = 1.4426950408889634074 / static_cast<double>(temperature);
        s.rh = r < FLT_MAX ? static_cast<float>(r) : FLT_MAX;
        s.rl = r < FLT_MAX ? static_cast<float>(r - static_cast<double>(s.rh)) : 0.0f;
    }

    // ---- the largest entry
    cluster_wait();
    if (by_list && !greedy)
        for (int c = 0; c < C; ++c) put(&s.maxima[rank * kThreads + tid], c, __float_as_uint(top_own));
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
    Scale sc;
    sc.top = -INFINITY;
    for (int c = 0; c < C; ++c) sc.top = fmaxf(sc.top, s.cta_max[c]);
    sc.rh = s.rh;
    sc.rl = s.rl;

    float* probs = a.probs != nullptr ? a.probs + static_cast<int64_t>(row) * a.ld_probs : nullptr;
    auto clear_probs = [&]() {
        if (probs == nullptr) return;
        const bool vec = (reinterpret_cast<uintptr_t>(probs + sl.begin) & 15u) == 0;
        const int n = sl.end - sl.begin;
        if (vec) {
            for (int i = tid; i < n / 4; i += kThreads)
                *reinterpret_cast<float4*>(probs + sl.begin + 4 * i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int i = n / 4 * 4 + tid; i < n; i += kThreads) probs[sl.begin + i] = 0.0f;
        } else {
            for (int i = tid; i < n; i += kThreads) probs[sl.begin + i] = 0.0f;
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

    // Entries that `pick` takes, to the first CTA's list; true if they fit (the same in every CTA).  The area of
    // maxima, bins and stage is free when it is called.
    auto collect = [&](auto pick) {
        __syncthreads();
        for (int st = 0; st < sl.steps(); ++st) {
            float x[kGroup];
            const int v = sl.read(st, x);
            bool any = false;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) any |= pick(x[i], v + i);
            if (!__any_sync(0xffffffffu, any)) continue;
            if (any) {
#pragma unroll 1
                for (int i = 0; i < kGroup; ++i) {
                    float z = x[0];
#pragma unroll
                    for (int j = 1; j < kGroup; ++j) z = i == j ? x[j] : z;
                    if (!pick(z, v + i)) continue;
                    const uint32_t at = atomicAdd(&s.stage_count, 1u);
                    if (at < kList) s.stage[at] = (static_cast<uint64_t>(order_key(z)) << 32) | ~static_cast<uint32_t>(v + i);
                }
            }
        }
        __syncthreads();
        const uint32_t n = s.stage_count;
        if (tid < C) put(&s.cta_count[rank], tid, n);
        if (tid == 0) s.stage_base = n > 0 ? add_remote(&s.list_count, 0, n) : 0;
        __syncthreads();
        const uint32_t base = s.stage_base;
        for (uint32_t i = tid; i < n; i += kThreads)
            if (i < kList && base + i < kList) put(&s.list[base + i], 0u, s.stage[i]);
        cluster_sync();
        uint32_t all = 0;
        for (int c = 0; c < C; ++c) all += s.cta_count[c];
        return all;
    };

    // smallest entry that min-p keeps
    float zmin = -INFINITY;
    if (use_m) {
        const double t = static_cast<double>(sc.top) + static_cast<double>(temperature) * log(static_cast<double>(fminf(m_in, 1.0f)));
        zmin = static_cast<float>(t);
        if (static_cast<double>(zmin) < t) zmin = nextafterf(zmin, INFINITY);
        zmin = fminf(zmin, sc.top);
    }

    bool listed = false;
    if (by_list) {
        // ---- a bound that at least k entries reach: the k-th largest of the threads' maxima, or a little less
        uint32_t key[kMaxCtas];
        uint32_t hi = order_key(sc.top) + 1, lo = 0;         // entries >= lo: at least k; >= hi: fewer
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c) key[c] = c < C ? order_key(s.maxima[c * kThreads + tid]) : 0;
        const uint32_t enough = static_cast<uint32_t>(k_in) + k_in / 8 + 8;
        int slot = 0;
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            uint32_t n = 0;
#pragma unroll
            for (int c = 0; c < kMaxCtas; ++c) n += key[c] >= mid ? 1u : 0u;
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) s.warp_sum[slot][warp] = n;
            __syncthreads();
            uint32_t total = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) total += static_cast<uint32_t>(s.warp_sum[slot][w]);
            slot ^= 1;
            if (total >= static_cast<uint32_t>(k_in)) {
                lo = mid;
                if (total <= enough) break;
            } else {
                hi = mid;
            }
        }
        const float bound = lo <= 0x007fffffu ? -INFINITY : key_value(lo);   // below every number: all of them
        clear_probs();
        const uint32_t n_all = collect([&](float z, int) { return z >= bound && z > -INFINITY; });
        listed = n_all <= kList;
        if (listed) {
            if (rank != 0) return;
            const int n = static_cast<int>(n_all), k = min(k_in, n);
            sort_list(s.list, n);
            uint64_t w[kPerThread], before[kPerThread];
            const uint64_t mass = list_masses(s, k, sc, w, before);
            const uint64_t limit = use_p ? max(scaled(p_in, mass, true), uint64_t(1)) : ~0ull;
            // how many of the sorted entries are kept, and their mass
            int kept = 0;
            uint64_t own = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const int at = tid * kPerThread + i;
                if (at < k && before[i] < limit && list_value(s.list[at]) >= zmin) {
                    ++kept;
                    own += w[i];
                }
            }
            __syncthreads();
            const uint64_t sum = block_sum64(s, own, 0);
            const int nk = static_cast<int>(block_sum64(s, static_cast<uint64_t>(kept), 1));
            const uint64_t target = scaled(u, sum, false);
            // the masses where `stage` was: every CTA has sent its own
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
                if (tid * kPerThread + i < nk) s.stage[tid * kPerThread + i] = w[i];
            __syncthreads();
            const Inverse inv = inverse(sum);
            int v = 0x7fffffff, last = -1;
            for (int i = tid; i < nk; i += kThreads) {
                const int idx = list_index(s.list[i]);
                if (probs != nullptr) probs[idx] = probability(list_value(s.list[i]), sc, s.pow, inv);
                if (s.stage[i] == 0) continue;
                last = max(last, idx);
                if (nk <= 512) {
                    uint64_t upto = 0;
                    for (int j = 0; j < nk; ++j) upto += list_index(s.list[j]) <= idx ? s.stage[j] : 0;
                    if (upto > target) v = min(v, idx);
                }
            }
            if (nk > 512) {
                // the least index up to which more than the target lies
                int below = -1, at = a.V - 1;
                while (at - below > 1) {
                    const int mid = below + (at - below) / 2;
                    uint64_t upto = 0;
                    for (int i = tid; i < nk; i += kThreads) upto += list_index(s.list[i]) <= mid ? s.stage[i] : 0;
                    if (block_sum64(s, upto, slot) > target) at = mid; else below = mid;
                    slot ^= 1;
                }
                v = sum > target ? at : 0x7fffffff;
            }
            v = __reduce_min_sync(0xffffffffu, v);
            last = __reduce_max_sync(0xffffffffu, last);
            __syncthreads();
            if (lane == 0) s.warp_sum[0][warp] = (static_cast<uint64_t>(static_cast<uint32_t>(v)) << 32) | static_cast<uint32_t>(last + 1);
            __syncthreads();
            if (tid == 0) {
                for (int i = 0; i < kWarps; ++i) {
                    v = min(v, static_cast<int>(s.warp_sum[0][i] >> 32));
                    last = max(last, static_cast<int>(static_cast<uint32_t>(s.warp_sum[0][i])) - 1);
                }
                a.tokens[row] = v != 0x7fffffff ? v : last;  // u of 1 or more: the last one kept
            }
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
    if (use_k) cut = narrow(cut, false, static_cast<uint64_t>(k_in));
    if (use_p) {
        // ---- masses of bins of z, largest first
        __syncthreads();
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = make_uint2(0u, 0u);
        if (tid == 0) s.stage_count = 0;
        if (rank == 0 && tid == 0) s.list_count = 0;
        __syncthreads();
        auto bin_of = [&](float z) { return min(kBins - 1, static_cast<int>(fminf((sc.top - z) * sc.rh * kBinsPerOctave, 1.0e6f))); };
        sl.each([&](float z, int v) {
            if (!cut.keeps(z, v)) return;
            const uint64_t w = weight(z, sc, s.pow);
            if (w == 0) return;
            uint2* h = &s.hist[bin_of(z)];
            const uint32_t wl = static_cast<uint32_t>(w), old = atomicAdd(&h->x, wl);
            const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
            if (wh != 0u) atomicAdd(&h->y, wh);
        });
        cluster_sync();
        // this CTA's share of the bins: sums over the cluster, then the mass of the share to every CTA
        const int share = kBins / C, b0 = static_cast<int>(rank) * share;      // C is a power of two
        uint64_t own[kBins / kThreads];
        uint64_t mine = 0;
        const int each = (share + kThreads - 1) / kThreads;
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) {
            own[i] = 0;
            const int b = tid * each + i;
            if (i < each && b < share)
                for (int c = 0; c < C; ++c) {
                    const uint2 h = get2(&s.hist[b0 + b], c);
                    own[i] += (static_cast<uint64_t>(h.y) << 32) | h.x;
                }
            mine += own[i];
        }
        const int now = flip;
        const uint64_t mass = cluster_sum(mine);
        uint64_t before = 0;
        for (int c = 0; c < static_cast<int>(rank); ++c) before += s.cta_sum[now][c];
        for (int w = 0; w < warp; ++w) before += s.warp_sum[now][w];
        before += warp_scan64(mine, lane) - mine;
        const uint64_t limit = max(scaled(p_in, mass, true), uint64_t(1));
        // the bin of the last entry before which less than the limit lies: mass up to it reaches the limit
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) {
            if (own[i] != 0 && before < limit && before + own[i] >= limit)
                for (int c = 0; c < C; ++c) {
                    put(&s.bin, c, static_cast<uint32_t>(b0 + tid * each + i));
                    put(&s.bin_before, c, before);
                }
            before += own[i];
        }
        cluster_sync();
        const int bin = s.bin;
        const uint64_t bin_before = s.bin_before;
        const uint32_t n = collect([&](float z, int v) { return z > -INFINITY && bin_of(z) == bin && cut.keeps(z, v); });
        if (n <= kList) {
            if (rank == 0) {
                sort_list(s.list, static_cast<int>(n));
                uint64_t w[kPerThread], b[kPerThread];
                list_masses(s, static_cast<int>(n), sc, w, b);
#pragma unroll
                for (int i = 0; i < kPerThread; ++i) {
                    const int at = tid * kPerThread + i;
                    // weights fall: the entry whose mass reaches the limit
                    if (w[i] != 0 && bin_before + b[i] < limit && bin_before + b[i] + w[i] >= limit)
                        for (int c = 0; c < C; ++c) {
                            put(&s.cut_key, c, static_cast<uint32_t>(s.list[at] >> 32));
                            put(&s.cut_index, c, static_cast<uint32_t>(list_index(s.list[at])));
                        }
                }
            }
            cluster_sync();
            cut = Cut{key_value(s.cut_key), s.cut_index};
        } else {
            cut = narrow(cut, true, limit);
        }
    }
    if (zmin > cut.z) cut = Cut{zmin, 0x7fffffff};

    // ---- the sum of what is kept, by warps; the warp with the border looks again
    uint64_t mine = 0;
    sl.each([&](float z, int v) {
        if (cut.keeps(z, v)) mine += weight(z, sc, s.pow);
    });
    const uint64_t in_warp = warp_sum64(mine);
    const int now = flip;
    __syncthreads();
    const uint64_t sum = cluster_sum(mine);
    const uint64_t target = min(scaled(u, sum, false), sum - 1);       // u of 1 or more: the last one kept
    uint64_t before = 0;
    for (int c = 0; c < static_cast<int>(rank); ++c) before += s.cta_sum[now][c];
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
        const Inverse inv = inverse(sum);
        for (int g = sl.g0 + lane; g < sl.g1; g += 32) {
            float x[kGroup];
            Slice<E>::unpack(sl.data[g], x);
            const int v = sl.group_index(g);
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                if (v + i >= sl.begin && v + i < sl.end)
                    probs[v + i] = cut.keeps(x[i], v + i) ? probability(x[i], sc, s.pow, inv) : 0.0f;
        }
    }
    // no CTA leaves while another may still write into or read from its shared memory
    cluster_sync();
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
    // the probabilities may not lie over the logits: a CTA writes its own while others still read
    if (probs != nullptr) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(probs);
        const uintptr_t nx = (static_cast<uintptr_t>(R - 1) * ld + V) * align, ny = (static_cast<uintptr_t>(R - 1) * ld_probs + V) * 4;
        if (x < y + ny && y < x + nx) return DSA_ERR_INVALID_ARG;
    }
    int ctas = 1;
    while (ctas < kMaxCtas && V > ctas * 2048) ctas *= 2;
    const int slice = ((V + ctas - 1) / ctas + 7) / 8 * 8;
    const size_t smem = sizeof(SampleShared) + (static_cast<size_t>(slice) * align + 15) / 16 * 16 + 16;
    SampleArgs a{logits, ld, V, temperature, top_k, top_p, min_p, u, tokens, probs, ld_probs, ctas, slice, dev_err};
    const void* kernel = bf16 ? reinterpret_cast<const void*>(&sample_tokens_kernel<uint16_t>)
                              : reinterpret_cast<const void*>(&sample_tokens_kernel<float>);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return DSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(R) * ctas);
    cfg.blockDim = dim3(kThreads);
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
