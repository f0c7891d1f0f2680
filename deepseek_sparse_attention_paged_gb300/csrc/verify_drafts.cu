// verify_drafts.cu -- acceptance of drafted tokens against the target's probabilities, and the draw
// of the token that follows the last accepted one, from given random numbers.
//
// Mathematics (rejection sampling of speculative decoding; Leviathan et al. 2023): row j of a
// request holds the target distribution p after its j-th token, x_j the token drafted there and q
// the draft's distribution.  x_j is accepted while u_j q(x_j) < p(x_j); at the first row where it is
// not, the next token is drawn from w = max(p - q, 0) (after the last draft: w = p) by inverting its
// cumulative sum: the least v with sum_{i <= v} w_i > u_s sum_i w_i.
//
// Sums: the drawn token must not depend on how the sum is split, so every sum is an unevaluated pair of
// fp32 numbers (about 47 bits), the difference p - q included.  fp64 would do the same, but its unit here
// is slow enough to be felt: with it one request took 14 us.  Adding in fp32 would move the borders by
// about 2^-24 of the sum each.
//
// One cluster of 8 CTAs per request, each with an eighth of the vocabulary: only the one row of p
// and of q that the draw needs is read, once, with all group sums kept in shared memory; the CTAs
// swap their totals through distributed shared memory, and the CTA whose range holds the border
// re-reads one group of 512 entries.
//
// Bound by the chain of dependent steps (acceptance, sums, totals across the cluster, border), about 7 us.  Measured:
// 1 request 7.9 us, 8 of 131072 entries 11.2 us, 64 of them 18.6 us with the inputs in HBM (the read of 49 MB alone
// 7.2 us at the copy rate; 16.6 us when L2 holds it).
#include "dsa_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCtas = 8;                 // cluster size: CTAs per request
constexpr int kGroup = 512;                    // entries per recorded sum: 4 steps x 32 lanes x 4
constexpr int kMaxVocab = 1 << 24;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The two halves of a cluster barrier: what comes between needs no peer.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A sum hi + lo, |lo| at most half a unit of hi.
struct Sum {
    float hi, lo;
};

__device__ __forceinline__ Sum normal(float hi, float lo) {
    const float h = __fadd_rn(hi, lo);
    return Sum{h, __fsub_rn(lo, __fsub_rn(h, hi))};
}
__device__ __forceinline__ Sum operator+(Sum a, Sum b) {
    const float s = __fadd_rn(a.hi, b.hi);
    return normal(s, __fadd_rn(two_sum_err(a.hi, b.hi, s), __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ bool operator>(Sum a, Sum b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Sum shfl_up(Sum v, int d) {
    return Sum{__shfl_up_sync(0xffffffffu, v.hi, d), __shfl_up_sync(0xffffffffu, v.lo, d)};
}
__device__ __forceinline__ Sum shfl(Sum v, int l) {
    return Sum{__shfl_sync(0xffffffffu, v.hi, l), __shfl_sync(0xffffffffu, v.lo, l)};
}
// Inclusive prefix sums over the lanes.  Rolled: code that runs once or twice costs its instruction fetches
// (unrolled, the last steps of the draw took 5200 cycles).
__device__ __forceinline__ Sum scan(Sum v, int lane) {
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const Sum o = shfl_up(v, d);
        if (lane >= d) v = o + v;
    }
    return v;
}

// Store a sum at the same shared-memory offset in CTA `rank` of the cluster, counted as 8 transaction
// bytes on the barrier at `bar`'s offset there (the receiver's wait on it orders the data).
__device__ __forceinline__ void send_sum(Sum* p, uint64_t* bar, uint32_t rank, Sum v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_addr(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(ptx::smem_addr(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(a), "f"(v.hi),
                 "f"(v.lo), "r"(b)
                 : "memory");
}

// How the row's weights are formed from p and q.
enum Mode { kPlain = 0, kResidual = 1, kWithout = 2 };   // w = p; w = max(p - q, 0); w = p with entry x zeroed

// Four consecutive entries v .. v + 3 of the row (entries past V are 0); for kWithout q = p at x.
template <bool VEC>
__device__ __forceinline__ void load4(const float* __restrict__ p_row, const float* __restrict__ q_row, int mode, int x,
                                      int v, int V, float (&p)[4], float (&q)[4]) {
    if (VEC && v + 4 <= V) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p_row + v));
        p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
        if (mode == kResidual) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(q_row + v));
            q[0] = b.x; q[1] = b.y; q[2] = b.z; q[3] = b.w;
        } else {
            q[0] = q[1] = q[2] = q[3] = 0.0f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = v + e < V ? __ldg(p_row + v + e) : 0.0f;
            q[e] = (mode == kResidual && v + e < V) ? __ldg(q_row + v + e) : 0.0f;
        }
    }
    if (mode == kWithout) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (v + e == x) p[e] = 0.0f;
    }
}

// max(p - q, 0), exact; an entry counts when it is positive and finite.
__device__ __forceinline__ Sum weight(float p, float q) {
    const float d = __fsub_rn(p, q);
    const float e = __fsub_rn(__fsub_rn(p, d), q);   // exact for p >= q >= 0
    return d > 0.0f && d < INFINITY ? Sum{d, e} : Sum{0.0f, 0.0f};
}

template <bool VEC>
__global__ void __launch_bounds__(kVerifyThreads) __cluster_dims__(kVerifyCtas, 1, 1)
verify_drafts_kernel(const float* __restrict__ target, int64_t ld_t, const float* __restrict__ draft, int64_t ld_d,
                     int V, const int32_t* __restrict__ tokens, const int32_t* __restrict__ cu_q, int T,
                     const float* __restrict__ u_accept, const float* __restrict__ u_sample,
                     int32_t* __restrict__ out_tokens, int32_t* __restrict__ accepted, int32_t* err) {
    extern __shared__ Sum group_sum[];           // [groups of this CTA]: sums, then inclusive prefix sums
    __shared__ Sum totals[2][kVerifyCtas];        // per pass over the row: every CTA's sum
    __shared__ uint64_t totals_full[2];
    __shared__ int s_first, s_x;
    ptx::griddep_wait();                         // a programmatic dependent: what came before is complete
    const int b = blockIdx.x / kVerifyCtas;
    const int rank = static_cast<int>(cluster_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = max(0, min(T, __ldg(cu_q + b)));
    const int r1 = max(r0, min(T, __ldg(cu_q + b + 1)));
    const int n_draft = r1 - r0 - 1;
    if (rank == 0 && threadIdx.x == 0 && (r0 != __ldg(cu_q + b) || r1 != __ldg(cu_q + b + 1)))
        raise_error(err, DSA_DEVERR_INDEX_RANGE);
    if (n_draft < 0) {                           // no row: nothing to verify (uniform over the cluster)
        if (rank == 0 && threadIdx.x == 0) accepted[b] = 0;
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&totals_full[i], 1);
            ptx::mbar_arrive_expect_tx(&totals_full[i], kVerifyCtas * sizeof(Sum));
        }
        ptx::fence_barrier_init();
    }
    __syncthreads();
    cluster_arrive();                            // every CTA's barriers exist before any writes into its shared memory
    // ---- acceptance: the first row whose draft is missing or rejected (every CTA finds it for itself)
    if (warp == 0) {
        int first = n_draft, x_first = -1;
        for (int j0 = 0; j0 < n_draft; j0 += 32) {
            const int j = j0 + lane;
            bool stop = false;
            int x = -1;
            if (j < n_draft) {
                x = __ldg(tokens + r0 + j);
                if (x >= V) {
                    if (rank == 0) raise_error(err, DSA_DEVERR_INDEX_RANGE);
                    x = -1;
                }
                stop = true;
                if (x >= 0) {
                    const float p = __ldg(target + static_cast<int64_t>(r0 + j) * ld_t + x);
                    const float q = draft != nullptr ? __ldg(draft + static_cast<int64_t>(r0 + j) * ld_d + x) : 1.0f;
                    // u q < p without rounding: the product of two fp32 numbers is exact in fp64, subnormal ones
                    // included (in fp32 the error of a product below 2^-102 is itself cut off)
                    stop = !(static_cast<double>(__ldg(u_accept + r0 + j)) * static_cast<double>(q) < static_cast<double>(p));
                }
            }
            const uint32_t m = __ballot_sync(0xffffffffu, stop);
            if (m != 0u) {
                first = j0 + __ffs(m) - 1;
                x_first = __shfl_sync(0xffffffffu, x, __ffs(m) - 1);
                break;
            }
        }
        if (lane == 0) {
            s_first = first;
            s_x = x_first;
        }
    }
    __syncthreads();
    const int first = s_first, x = s_x;
    if (rank == 0) {
        for (int j = threadIdx.x; j < r1 - r0; j += kVerifyThreads)
            if (j != first) out_tokens[r0 + j] = j < first ? __ldg(tokens + r0 + j) : -1;
        if (threadIdx.x == 0) accepted[b] = first;
    }
    // ---- the draw
    const float* p_row = target + static_cast<int64_t>(r0 + first) * ld_t;
    const float* q_row = draft != nullptr ? draft + static_cast<int64_t>(r0 + first) * ld_d : nullptr;
    const int groups_all = (V + kGroup - 1) / kGroup;
    const int per_cta = (groups_all + kVerifyCtas - 1) / kVerifyCtas;
    const int g_begin = min(groups_all, rank * per_cta), g_end = min(groups_all, g_begin + per_cta);
    const int ng = g_end - g_begin;
    int mode = x < 0 ? kPlain : (q_row != nullptr ? kResidual : kWithout);
    int pass = 0;
    bool late = false, mass = false;
    const uint64_t deadline = ptx::wait_deadline();
    for (;;) {
        for (int g = warp; g < ng; g += kVerifyWarps) {
            float hi = 0.0f, lo = 0.0f;
            float p[4][4], q[4][4];
            const int v0 = (g_begin + g) * kGroup + lane * 4;
#pragma unroll
            for (int s = 0; s < 4; ++s) load4<VEC>(p_row, q_row, mode, x, v0 + s * 128, V, p[s], q[s]);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Sum w = weight(p[s][e], q[s][e]);
                    const float t = __fadd_rn(hi, w.hi);
                    lo = __fadd_rn(lo, __fadd_rn(two_sum_err(hi, w.hi, t), w.lo));
                    hi = t;
                }
            Sum sum = normal(hi, lo);
#pragma unroll 1
            for (int m = 16; m > 0; m >>= 1)
                sum = sum + Sum{__shfl_xor_sync(0xffffffffu, sum.hi, m), __shfl_xor_sync(0xffffffffu, sum.lo, m)};
            if (lane == 0) group_sum[g] = sum;
        }
        __syncthreads();
        if (pass == 0) cluster_wait();
        if (warp == 0) {                         // inclusive prefix sums of this CTA's groups
            Sum carry{0.0f, 0.0f};
            for (int g0 = 0; g0 < ng; g0 += 32) {
                const Sum v = carry + scan(g0 + lane < ng ? group_sum[g0 + lane] : Sum{0.0f, 0.0f}, lane);
                if (g0 + lane < ng) group_sum[g0 + lane] = v;
                carry = shfl(v, 31);
            }
            if (lane < kVerifyCtas) send_sum(&totals[pass][rank], &totals_full[pass], lane, carry);
        }
        if (!ptx::mbar_wait(&totals_full[pass], 0, deadline)) late = true;
        if (__syncthreads_or(late)) {            // all leave together
            if (threadIdx.x == 0) {              // no token, whichever CTA would have drawn it
                out_tokens[r0 + first] = -1;
                raise_error(err, DSA_DEVERR_TIMEOUT);
            }
            cluster_arrive();                    // not before every CTA that may still send has left or come here
            cluster_wait();
            return;
        }
        for (int c = 0; c < kVerifyCtas; ++c) mass |= totals[pass][c].hi > 0.0f;
        if (mass || mode == kPlain) break;
        mode = kPlain;                           // p <= q everywhere: draw from p itself, in a second pass
        ++pass;
    }
    if (warp != 0) return;
    // the same sums in every CTA (lane c: CTA c's): base of this CTA, total, owner of the border
    const Sum part = lane < kVerifyCtas ? totals[pass][lane] : Sum{0.0f, 0.0f};
    const Sum upto = scan(part, lane);
    const Sum all = shfl(upto, 31);
    const Sum before = shfl(upto, max(rank - 1, 0));
    const Sum base = rank > 0 ? before : Sum{0.0f, 0.0f};
    const float u = __ldg(u_sample + b);
    const float ua = __fmul_rn(u, all.hi);
    const Sum t = normal(ua, __fmaf_rn(u, all.lo, __fmaf_rn(u, all.hi, -ua)));
    const uint32_t with_mass = __ballot_sync(0xffffffffu, part.hi > 0.0f);
    const uint32_t past = __ballot_sync(0xffffffffu, part.hi > 0.0f && upto > t);
    // u outside [0, 1): the last entry with mass
    const int owner = past != 0u ? __ffs(past) - 1 : 31 - __clz(with_mass);   // -1: no mass
    if (owner < 0) {                             // a row without mass
        if (rank == 0 && lane == 0) {
            out_tokens[r0 + first] = -1;
            raise_error(err, DSA_DEVERR_PROB);
        }
        return;
    }
    if (rank != owner) return;
    // the first group whose prefix passes t (the last with mass if none does)
    int g_hit = -1, g_last = -1;
    for (int g0 = 0; g0 < ng; g0 += 32) {
        const int g = g0 + lane;
        const Sum inc = g < ng ? group_sum[g] : Sum{0.0f, 0.0f};
        const Sum exc = (g < ng && g > 0) ? group_sum[g - 1] : Sum{0.0f, 0.0f};
        const bool some = g < ng && inc > exc;
        const uint32_t hit = __ballot_sync(0xffffffffu, some && base + inc > t);
        const uint32_t any = __ballot_sync(0xffffffffu, some);
        if (any != 0u) g_last = g0 + 31 - __clz(any);
        if (hit != 0u) {
            g_hit = g0 + __ffs(hit) - 1;
            break;
        }
    }
    if (g_hit < 0) g_hit = max(g_last, 0);
    Sum run = g_hit > 0 ? base + group_sum[g_hit - 1] : base;
    // the first of 32 runs of 16 entries whose prefix passes t, and in it the first entry; where the border
    // lies within the rounding of a sum, the last one with mass
    int v0 = (g_begin + g_hit) * kGroup;
    int token = -1;
#pragma unroll 1
    for (int len = kGroup / 32; len > 0; len = len > 1 ? 1 : 0) {
        const int v = v0 + lane * len;                 // len = 16: a run each; len = 1: an entry each of the run
        Sum own{0.0f, 0.0f};
        if (len > 1) {
#pragma unroll 1
            for (int e = 0; e < len; e += 4) {
                float p[4], q[4];
                load4<VEC>(p_row, q_row, mode, x, v + e, V, p, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) own = own + weight(p[i], q[i]);
            }
        } else if (lane < kGroup / 32) {               // one entry at any address: no vector load
            float p[4], q[4];
            load4<false>(p_row, q_row, mode, x, v, min(V, v + 1), p, q);
            own = weight(p[0], q[0]);
        }
        const Sum upto = scan(own, lane);
        const uint32_t some = __ballot_sync(0xffffffffu, own.hi > 0.0f);
        const uint32_t over = __ballot_sync(0xffffffffu, own.hi > 0.0f && run + upto > t);
        if (some == 0u) break;                         // unreachable: the group has mass
        const int l = over != 0u ? __ffs(over) - 1 : 31 - __clz(some);
        const Sum before_l = shfl(upto, max(l - 1, 0));
        if (l > 0) run = run + before_l;
        v0 += l * len;
        if (len == 1) token = v0;
    }
    if (lane == 0) out_tokens[r0 + first] = token;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_verify_drafts(const float* target_probs, int64_t target_ld, const float* draft_probs,
                                        int64_t draft_ld, int32_t V, const int32_t* draft_tokens, const int32_t* cu_q,
                                        int32_t B, int32_t T, const float* accept_u, const float* sample_u,
                                        int32_t* out_tokens, int32_t* accepted, int32_t* dev_err, void* stream) {
    using namespace dsa;
    if (B < 0 || T < 0 || V < 1) return DSA_ERR_INVALID_ARG;
    if (V > kMaxVocab || B > 0x7fffffff / kVerifyCtas) return DSA_ERR_UNSUPPORTED;
    if (B == 0) return DSA_OK;
    if (!cu_q || !accepted) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!target_probs || !draft_tokens || !accept_u || !sample_u || !out_tokens)) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (target_ld < V || (draft_probs != nullptr && draft_ld < V))) return DSA_ERR_INVALID_ARG;
    // every CTA of a cluster reads the drafts, and of other requests at any time: the output may not lie over them
    const uintptr_t in_at = reinterpret_cast<uintptr_t>(draft_tokens), out_at = reinterpret_cast<uintptr_t>(out_tokens);
    const uintptr_t in_bytes = static_cast<uintptr_t>(T) * sizeof(int32_t);
    if (T > 0 && in_at < out_at + in_bytes && out_at < in_at + in_bytes) return DSA_ERR_INVALID_ARG;
    const bool vec = aligned16(target_probs) && target_ld % 4 == 0 &&
                     (draft_probs == nullptr || (aligned16(draft_probs) && draft_ld % 4 == 0));
    const int groups = (V + kGroup - 1) / kGroup;
    const size_t smem = static_cast<size_t>((groups + kVerifyCtas - 1) / kVerifyCtas) * sizeof(Sum);   // <= 32 KB
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * kVerifyCtas);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, vec ? verify_drafts_kernel<true> : verify_drafts_kernel<false>, target_probs, target_ld,
                           draft_probs, draft_ld, V, draft_tokens, cu_q, T, accept_u, sample_u, out_tokens, accepted,
                           dev_err) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}
