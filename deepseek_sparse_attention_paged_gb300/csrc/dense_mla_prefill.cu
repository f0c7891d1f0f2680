// dense_mla_prefill.cu -- attention of a prompt in expanded form (sm_103a): per-head keys and values
// made from the latent rows, one rope key shared by all heads.
//
// Follows vllm mla/common.py, MLACommonImpl._forward_prefill (k = [k_nope, k_pe], causal attention
// over ragged requests) and _compute_prefill_context (a chunk's queries over earlier keys).
//
// Mathematics: S_ij = scale (<q_i[0:128], k_nope_j> + <q_i[128:192], k_pe_j>), O = softmax(S) V, in
// one pass over the keys with a running maximum m and sum l per query: P = 2^(c S - c m)
// (c = scale log2 e), O = sum P V, out = O / l.  m only moves when a tile's maximum exceeds it by
// more than 8 / c (then O and l are rescaled); P < 2^8 otherwise.  S, m, l and O are fp32; P is
// rounded to bf16 for its product with V (the tensor cores take no wider A operand at this rate),
// l sums the unrounded P.
//
// Bound: the tensor cores.  640 FLOP per (query, key, head); a 128 x 128 tile is 768 cycles of
// Q K^T (K = 192) and 512 of P V at 8192 FLOP per cycle and SM, its softmax 16384 exponentials
// (512 to 1024 cycles of the special-function unit).  So a CTA holds two tiles of 128 queries of
// one head and one request: while the softmax warps of one work, the tensor cores run the other's
// products.
//
// CTA: block qb of 256 query rows of request b, head h.  Roles (384 threads):
//   warps 0-3, 4-7  softmax of query tile 0 / 1: one thread per query (TMEM lane), 128 scores in
//                   registers, P written back over the scores as bf16; O / l at the end;
//   warp 8          TMA: the query tiles, then K (two 64-dim slabs of k_nope, one of k_pe) and V
//                   (two slabs) of each 128-key tile through a ring of eight 16 KB slabs;
//   warp 9          MMA: S = Q K^T with both operands in shared memory, O += P V with P in tensor
//                   memory, alternating between the query tiles.
// Tensor memory (512 columns): S / P of tile 0, of tile 1, O of tile 0, of tile 1 (128 each).
// Shared memory: queries 96 KB, ring 128 KB.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace dsa {
namespace {

using namespace attn;

constexpr int kTileQ = 128, kTileK = 128, kBlockQ = 2 * kTileQ;
constexpr int kSlabBytes = 128 * 128;                     // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kRing = 8;
constexpr int kQSlabs = 3, kKSlabs = 3, kVSlabs = 2;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kPreThreads = 384;                          // three warpgroups; warps 10 and 11 only fill the third
constexpr int kSoftmaxRegs = 192, kOtherRegs = 112;       // 2 x 128 x 192 + 128 x 112 <= 384 x 168 at launch
constexpr uint32_t kColS = 0, kColO = 256;                // + 128 * tile
constexpr size_t kPreSmem = 1024 + size_t(2 * kQSlabs + kRing) * kSlabBytes + 512;
static_assert(kPreSmem <= 232448, "shared-memory budget");

struct PreBars {
    uint64_t q_full[2];
    uint64_t full[kRing], empty[kRing];
    uint64_t s_full[2];      // scores of the tile's next step complete (and with them its previous P V)
    uint64_t p_full[2];      // P written (4 softmax warps)
    uint64_t o_full[2];      // last P V complete
    uint32_t tmem_slot;
    int item[4];             // request, query block, first query row, queries of the request
};
static_assert(sizeof(PreBars) <= 512, "barrier block");

// The CTA's work: block x in the order of requests, the last (longest) query block of each first.
__device__ __forceinline__ void find_item(const int32_t* __restrict__ cu_q, int B, int T, int x, int lane, int* item,
                                          int32_t* err) {
    int carry = 0;
    bool found = false;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        int q0 = 0, nq = 0;
        if (b < B) {
            const int lo = __ldg(cu_q + b), hi = __ldg(cu_q + b + 1);
            q0 = max(0, min(T, lo));
            nq = max(0, min(T, hi) - q0);
            if (x == 0 && (lo < 0 || hi > T)) raise_error(err, DSA_DEVERR_INDEX_RANGE);
        }
        const int nb = (nq + kBlockQ - 1) / kBlockQ;
        int inc = nb;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, x < carry + inc);
        if (!found && hit != 0u) {
            found = true;
            if (lane == __ffs(hit) - 1) {
                item[0] = b;
                item[1] = nb - 1 - (x - (carry + inc - nb));
                item[2] = q0;
                item[3] = nq;
            }
            if (x != 0) return;                                // block 0 goes on to check every range
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
    }
}

__global__ void __launch_bounds__(kPreThreads, 1)
dense_mla_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap vmap,
                         const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int B, int T, int S, int H,
                         float scale, int causal, uint16_t* __restrict__ out, int64_t out_row, int64_t out_head,
                         float* __restrict__ lse_out, int32_t* err) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    unsigned char* qs = base;                                  // [2 tiles][3 slabs]
    unsigned char* ring = base + 2 * kQSlabs * kSlabBytes;     // [8]
    PreBars& bar = *reinterpret_cast<PreBars*>(ring + kRing * kSlabBytes);

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int h = blockIdx.y;
    if (warp == 0) {
        if (lane == 0) bar.item[0] = -1;
        __syncwarp();
        find_item(cu_q, B, T, static_cast<int>(blockIdx.x), lane, bar.item, err);
    } else if (warp == kTmaWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bar.q_full[i], 1);
            ptx::mbar_init(&bar.s_full[i], 1);
            ptx::mbar_init(&bar.p_full[i], 4);
            ptx::mbar_init(&bar.o_full[i], 1);
        }
        for (int s = 0; s < kRing; ++s) {
            ptx::mbar_init(&bar.full[s], 1);
            ptx::mbar_init(&bar.empty[s], 1);
        }
        ptx::fence_barrier_init();
    }
    __syncthreads();
    const int b = uniform(bar.item[0]);
    if (b < 0) return;                                         // past the last block (uniform)
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&bar.tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    const int qb = uniform(bar.item[1]), q0 = uniform(bar.item[2]), nq = uniform(bar.item[3]);
    const int k_lo = uniform(__ldg(cu_k + b)), k_hi = uniform(__ldg(cu_k + b + 1));
    const int k0 = max(0, min(S, k_lo));
    const int nk = max(0, min(S, k_hi) - k0);
    if (threadIdx.x == 0 && (k_lo < 0 || k_hi > S)) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    const int off = causal ? nk - nq : 0;                      // query i sees keys [0, off + i] (causal)
    // key tiles that tile i's rows see
    int n_tiles[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int first = qb * kBlockQ + i * kTileQ;
        const int last = min(nq, first + kTileQ) - 1;
        const int seen = last < first ? 0 : (causal ? max(0, min(nk, off + last + 1)) : nk);
        n_tiles[i] = (seen + kTileK - 1) / kTileK;
    }
    const int n = max(n_tiles[0], n_tiles[1]);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem_slot);
    const uint64_t deadline = ptx::wait_deadline();
    bool timed_out = false;

    if (warp >= kTmaWarp) {
        set_regs_dec<kOtherRegs>();
        if (warp == kTmaWarp) {
            // ---------------------------------------------------------------- TMA
            if (lane == 0 && n > 0) {
                uint32_t c = 0;                                    // slabs issued
                auto next = [&]() -> unsigned char* {              // the ring's next slab, once it is free
                    const int s = static_cast<int>(c % kRing);
                    if (!ptx::mbar_wait(&bar.empty[s], ((c / kRing) & 1u) ^ 1u, deadline)) timed_out = true;
                    if (timed_out) return nullptr;
                    ptx::mbar_arrive_expect_tx(&bar.full[s], kSlabBytes);
                    ++c;
                    return ring + s * kSlabBytes;
                };
                auto bar_of_last = [&]() { return &bar.full[(c - 1) % kRing]; };
                auto load_q = [&](int i) {
                    if (n_tiles[i] == 0) return;
                    ptx::mbar_arrive_expect_tx(&bar.q_full[i], kQSlabs * kSlabBytes);
                    for (int j = 0; j < kQSlabs; ++j)
                        ptx::tma_load_3d(qs + (i * kQSlabs + j) * kSlabBytes, &qmap, &bar.q_full[i], 64 * j, h,
                                         q0 + qb * kBlockQ + i * kTileQ);
                };
                auto load_k = [&](int t) {
                    for (int j = 0; j < kKSlabs && !timed_out; ++j)
                        if (unsigned char* dst = next()) {
                            if (j < 2) ptx::tma_load_3d(dst, &kmap, bar_of_last(), 64 * j, h, k0 + t * kTileK);
                            else ptx::tma_load_3d(dst, &pmap, bar_of_last(), 0, 0, k0 + t * kTileK);
                        }
                };
                load_q(0);
                load_k(0);
                load_q(1);
                for (int t = 0; t < n && !timed_out; ++t) {
                    for (int j = 0; j < kVSlabs && !timed_out; ++j)
                        if (unsigned char* dst = next())
                            ptx::tma_load_3d(dst, &vmap, bar_of_last(), 64 * j, h, k0 + t * kTileK);
                    if (t + 1 < n) load_k(t + 1);
                }
                // copies still in flight land before the CTA may leave (bounded)
                for (int i = 0; i < 2; ++i)
                    if (n_tiles[i] > 0 && !ptx::mbar_wait(&bar.q_full[i], 0, ptx::wait_deadline(20000000ull))) timed_out = true;
                for (uint32_t j = c > kRing ? c - kRing : 0; j < c; ++j)
                    if (!ptx::mbar_wait(&bar.full[j % kRing], (j / kRing) & 1u, ptx::wait_deadline(20000000ull)))
                        timed_out = true;
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- MMA
            constexpr uint32_t idesc_qk = ptx::instr_desc(1, 1, kTileQ, kTileK);
            constexpr uint32_t idesc_pv = ptx::instr_desc(1, 1, kTileQ, 128) | (1u << 16);   // B MN-major
            constexpr uint32_t idesc_pv_half = ptx::instr_desc(1, 1, kTileQ, 64) | (1u << 16);
            const uint32_t q_addr = ptx::smem_addr(qs), ring_addr = ptx::smem_addr(ring);
            // A wait that ran out only marks the step: the warp leaves together at the step's end.  What it
            // issues until then reads shared and tensor memory of this CTA only.
            bool late = false;
            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (!ptx::mbar_wait(b, parity, deadline)) late = true;
            };
            auto wait_slab = [&](uint32_t cc) { wait(&bar.full[cc % kRing], (cc / kRing) & 1u); };
            auto release = [&](uint32_t c0, int cnt) {         // free once the MMAs issued so far completed
                if (elect_one())
                    for (int j = 0; j < cnt; ++j) ptx::umma_commit(&bar.empty[(c0 + j) % kRing]);
            };
            // descriptors differ in their start address only (low word, 16-byte units): one add each
            const uint64_t q_desc = desc_sw128(q_addr, 16, 1024);
            const uint64_t k_desc = desc_sw128(ring_addr, 16, 1024), v_desc = desc_sw128(ring_addr, kSlabBytes, 1024);
            auto slab = [&](uint32_t cc) { return (cc % kRing) * (kSlabBytes / 16); };
            // S_i = Q_i K^T from the slabs at c0; the first user of a key tile waits for each slab in turn
            auto issue_s = [&](int i, uint32_t c0, bool first) {
                const uint64_t a = q_desc + i * (kQSlabs * kSlabBytes / 16);
#pragma unroll
                for (int j = 0; j < kKSlabs; ++j) {
                    if (first) {
                        wait_slab(c0 + j);
                        __syncwarp();
                        ptx::tc_fence_after_sync();
                    }
                    if (elect_one()) {
                        const uint64_t bk = k_desc + slab(c0 + j);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::umma_f16(tmem + kColS + 128 * i, a + (j * (kSlabBytes / 16) + kk * 2), bk + kk * 2,
                                          idesc_qk, (j | kk) != 0 ? 1u : 0u);
                        if (j == kKSlabs - 1) ptx::umma_commit(&bar.s_full[i]);
                    }
                }
            };
            // O_i += P_i V from the two slabs at c0
            auto issue_pv = [&](int i, uint32_t c0, uint32_t accumulate) {
                if (elect_one()) {
                    const uint64_t v0 = v_desc + slab(c0), v1 = v_desc + slab(c0 + 1);
                    const uint32_t o = tmem + kColO + 128 * i, p = tmem + kColS + 128 * i;
                    if (v1 > v0) {
#pragma unroll
                        for (int ks = 0; ks < kTileK / 16; ++ks)
                            umma_f16_ts(o, p + ks * 8, v0 + ks * 128, idesc_pv, ks != 0 ? 1u : accumulate);
                    } else {                                   // the ring wraps between the two slabs
#pragma unroll
                        for (int ks = 0; ks < kTileK / 16; ++ks) {
                            umma_f16_ts(o, p + ks * 8, v0 + ks * 128, idesc_pv_half, ks != 0 ? 1u : accumulate);
                            umma_f16_ts(o + 64, p + ks * 8, v1 + ks * 128, idesc_pv_half, ks != 0 ? 1u : accumulate);
                        }
                    }
                }
            };
            if (n > 0) {
                bool first = true;
                for (int i = 0; i < 2; ++i) {
                    if (n_tiles[i] == 0) continue;
                    wait(&bar.q_full[i], 0);
                    issue_s(i, 0, first);
                    first = false;
                }
                release(0, kKSlabs);
            }
            for (int t = 0; t < n; ++t) {
                // ring order: K(0), V(0), K(1), V(1), ...; this step uses V(t) and K(t + 1)
                const uint32_t c_v = static_cast<uint32_t>(t) * (kKSlabs + kVSlabs) + kKSlabs, c_k = c_v + kVSlabs;
                const int last = t < n_tiles[1] ? 1 : 0;       // the last tile that uses V(t)
                bool first_v = true, first_k = true;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (t >= n_tiles[i]) continue;
                    if (first_v) {
                        first_v = false;
                        wait_slab(c_v);
                        wait_slab(c_v + 1);
                        const int valid = nk - t * kTileK;
                        if (valid < kTileK) {
                            // rows past the request's last key are another request's, or anything: their
                            // P is 0, but 0 times NaN or infinity is not
                            __syncwarp();
                            for (int e = lane; e < (kTileK - valid) * 8; e += 32) {
                                const int row = valid + (e >> 3);
#pragma unroll
                                for (int j = 0; j < kVSlabs; ++j)
                                    *reinterpret_cast<uint4*>(ring + ((c_v + j) % kRing) * kSlabBytes + row * 128 +
                                                              (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            ptx::fence_proxy_async_smem();
                        }
                    }
                    wait(&bar.p_full[i], t & 1);
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    issue_pv(i, c_v, t != 0 ? 1u : 0u);
                    if (i == last) release(c_v, kVSlabs);
                    if (t + 1 < n_tiles[i]) {
                        issue_s(i, c_k, first_k);
                        first_k = false;
                    } else if (elect_one()) {
                        ptx::umma_commit(&bar.o_full[i]);
                    }
                }
                if (t + 1 < n) release(c_k, kKSlabs);
                if (__any_sync(0xffffffffu, late)) break;
            }
            if (late) timed_out = true;
        }
    } else {
        set_regs_inc<kSoftmaxRegs>();
        // ---------------------------------------------------------------- softmax, epilogue
        const int i = warp >> 2;                               // query tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int row = qb * kBlockQ + i * kTileQ + (warp & 3) * 32 + lane;   // query of the request
        const uint32_t s_addr = tmem + lane_base + kColS + 128 * i;
        const uint32_t o_addr = tmem + lane_base + kColO + 128 * i;
        const float cs = scale * kLog2e;
        const uint64_t cs2 = f32x2(cs, cs);
        const int vis = row < nq ? (causal ? max(0, min(nk, off + row + 1)) : nk) : 0;
        // keys that every row of the warp's tile sees: tiles below it need no mask
        const int row0 = qb * kBlockQ + i * kTileQ;
        const int all_see = causal ? min(nk, off + row0 + 1) : nk;
        float m_run = -INFINITY, l_run = 0.0f;
        for (int t = 0; t < n_tiles[i]; ++t) {
            if (!ptx::mbar_wait(&bar.s_full[i], t & 1, deadline)) timed_out = true;
            timed_out = __any_sync(0xffffffffu, timed_out);
            if (timed_out) break;
            ptx::tc_fence_after_sync();
            uint32_t s[4][32];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) ptx::tmem_ld_32x32b_x32(s_addr + 32 * q4, s[q4]);
            ptx::tmem_wait_ld();
            if ((t + 1) * kTileK > all_see) {
                const int lim = vis - t * kTileK;
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * q4 + e >= lim) s[q4][e] = 0xff800000u;   // -inf
            }
            float mx4[4];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
                mx4[q4] = __uint_as_float(s[q4][0]);
#pragma unroll
                for (int e = 1; e < 32; ++e) mx4[q4] = fmaxf(mx4[q4], __uint_as_float(s[q4][e]));
            }
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            const bool grow = (mx - m_run) * cs > kRescaleThreshold || (m_run == -INFINITY && mx > -INFINITY);
            if (__any_sync(0xffffffffu, grow)) {
                const float alpha = grow ? (m_run == -INFINITY ? 0.0f : exp2f((m_run - mx) * cs)) : 1.0f;
                if (grow) m_run = mx;
                l_run *= alpha;
                if (t > 0) {                                   // P V (t - 1) has completed: s_full covers it
#pragma unroll 1
                    for (int cc = 0; cc < 128; cc += 32) {
                        uint32_t o[32];
                        ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st_x32(o_addr + cc, o);
                    }
                }
            }
            const float neg = m_run == -INFINITY ? 0.0f : -m_run * cs;
            const uint64_t neg2 = f32x2(neg, neg);
            uint64_t sum2 = f32x2(0.0f, 0.0f);
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float a, bb;
                    unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(s[q4][e]), __uint_as_float(s[q4][e + 1])), cs2, neg2), a, bb);
                    a = fast_exp2(a);
                    bb = fast_exp2(bb);
                    sum2 = add_f32x2(sum2, f32x2(a, bb));
                    pk[e / 2] = pack_bf16x2(a, bb);
                }
                tmem_st_x16(s_addr + 16 * q4, pk);
            }
            tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar.p_full[i]);
            float sa, sb;
            unpack_f32x2(sum2, sa, sb);
            l_run += sa + sb;
        }
        bool have_o = n_tiles[i] > 0 && !timed_out;
        if (have_o) {
            const bool got = ptx::mbar_wait(&bar.o_full[i], 0, deadline);
            have_o = __all_sync(0xffffffffu, got);
            if (!have_o) timed_out = true;
            ptx::tc_fence_after_sync();
        }
        const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        uint16_t* dst = out + static_cast<int64_t>(q0 + row) * out_row + static_cast<int64_t>(h) * out_head;
#pragma unroll 1
        for (int cc = 0; cc < 128; cc += 32) {
            uint32_t o[32];
            if (have_o) {
                ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                ptx::tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
            if (vis == 0) {                                    // a query that sees nothing: 0 (O may hold 0 x NaN)
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
            if (row < nq) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint4 w;
                    w.x = pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                    w.y = pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                    w.z = pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                    w.w = pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                    *reinterpret_cast<uint4*>(dst + cc + e) = w;
                }
            }
        }
        if (row < nq && lse_out != nullptr)
            lse_out[static_cast<int64_t>(q0 + row) * H + h] =
                l_run == 0.0f ? -INFINITY : (m_run * cs + log2f(l_run)) * kLn2;
    }
    if (timed_out) raise_error(err, DSA_DEVERR_TIMEOUT);
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

bool strides_ok(int64_t row, int64_t head, int64_t heads, int64_t width) {
    return row >= width && row % 8 == 0 && head % 8 == 0 && (heads == 1 || head >= width);
}

// No two (row, head) outputs share an element: rows enclose the heads or heads enclose the rows.
bool disjoint(int64_t row, int64_t head, int64_t rows, int64_t heads, int64_t width) {
    return row >= (heads - 1) * head + width || head >= (rows - 1) * row + width;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_dense_mla_prefill(const void* q_bf16, int64_t q_row_stride, int64_t q_head_stride,
                                            const void* k_nope_bf16, int64_t k_row_stride, int64_t k_head_stride,
                                            const void* k_pe_bf16, int64_t pe_row_stride, const void* v_bf16,
                                            int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_q,
                                            const int32_t* cu_k, int32_t B, int32_t T, int32_t S, int32_t H,
                                            float scale, uint32_t flags, void* out_bf16, int64_t out_row_stride,
                                            int64_t out_head_stride, float* lse, int32_t* dev_err, void* stream) {
    using namespace dsa;
    if (T < 0 || B < 0 || S < 0 || H < 0) return DSA_ERR_INVALID_ARG;
    if (flags & ~static_cast<uint32_t>(DSA_CAUSAL)) return DSA_ERR_INVALID_ARG;
    if (T == 0 || B == 0 || H == 0) return DSA_OK;
    if (!q_bf16 || !cu_q || !cu_k || !out_bf16) return DSA_ERR_INVALID_ARG;
    if (S > 0 && (!k_nope_bf16 || !k_pe_bf16 || !v_bf16)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_bf16) || !aligned16(k_nope_bf16) || !aligned16(k_pe_bf16) || !aligned16(v_bf16) ||
        !aligned16(out_bf16))
        return DSA_ERR_INVALID_ARG;
    if (!strides_ok(q_row_stride, q_head_stride, H, 192) || !strides_ok(out_row_stride, out_head_stride, H, 128) ||
        (S > 0 && (!strides_ok(k_row_stride, k_head_stride, H, 128) || !strides_ok(v_row_stride, v_head_stride, H, 128) ||
                   !strides_ok(pe_row_stride, 0, 1, 64))))
        return DSA_ERR_INVALID_ARG;
    if (!disjoint(out_row_stride, out_head_stride, T, H, 128)) return DSA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !(scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * H >= 0x7fffffffLL || H > 65535) return DSA_ERR_UNSUPPORTED;
    // tensor maps hold byte strides below 2^40
    const int64_t lim = int64_t(1) << 39;
    for (int64_t st : {q_row_stride, q_head_stride, k_row_stride, k_head_stride, pe_row_stride, v_row_stride, v_head_stride})
        if (st >= lim) return DSA_ERR_UNSUPPORTED;
    auto encode = attn::tensor_map_encoder();
    if (encode == nullptr) return DSA_ERR_CUDA;
    CUtensorMap qmap, kmap, pmap, vmap;
    const bool keys = S > 0;   // without keys no copy runs and the maps stand on the queries
    if (!attn::encode_bf16_3d(encode, &qmap, q_bf16, 192, H, T, q_head_stride, q_row_stride, 64, kTileQ) ||
        !attn::encode_bf16_3d(encode, &kmap, keys ? k_nope_bf16 : q_bf16, 128, H, keys ? S : T,
                              keys ? k_head_stride : q_head_stride, keys ? k_row_stride : q_row_stride, 64, kTileK) ||
        !attn::encode_bf16_3d(encode, &pmap, keys ? k_pe_bf16 : q_bf16, 64, 1, keys ? S : T,
                              keys ? pe_row_stride : q_row_stride, keys ? pe_row_stride : q_row_stride, 64, kTileK) ||
        !attn::encode_bf16_3d(encode, &vmap, keys ? v_bf16 : q_bf16, 128, H, keys ? S : T,
                              keys ? v_head_stride : q_head_stride, keys ? v_row_stride : q_row_stride, 64, kTileK))
        return DSA_ERR_CUDA;
    if (cudaFuncSetAttribute(dense_mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kPreSmem)) != cudaSuccess)
        return DSA_ERR_CUDA;
    const int64_t blocks = T / kBlockQ + std::min<int64_t>(B, T);   // >= the sum of the requests' blocks
    dense_mla_prefill_kernel<<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(H)), kPreThreads, kPreSmem,
                               static_cast<cudaStream_t>(stream)>>>(
        qmap, kmap, pmap, vmap, cu_q, cu_k, B, T, S, H, scale, (flags & DSA_CAUSAL) ? 1 : 0,
        static_cast<uint16_t*>(out_bf16), out_row_stride, out_head_stride, lse, dev_err);
    return launch_status();
}
