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
// products.  Measured: 8192 queries and keys, 19 heads, no mask 448 us (1.82 PFLOP/s; Q K^T reads both operands
// from shared memory, 8 KB an MMA, which takes 79 cycles for 64); causal with 128 heads 1.58 ms (1.78 one call
// after the other, at the power limit), with 16 heads 213 us; 8 prompts of 128 to 2048 362 us (84 % of their tiles'
// area counts); 1000 queries after 15001 keys 789 us, with 16 heads 115 us.
//
// Work item: block qb of 256 query rows of request b, head h; requests in the caller's order, of each the longest
// block first, over a group of heads whose keys and values fit L2.  The grid has one block per item; a CTA
// takes over the items of blocks that have not started (cluster launch control) until none is left, so
// that an item's first copies and scores run while the one before is still at its last step and its output.
// Calls with few items split each one's keys over a cluster of C = 2 or 4 CTAs instead (one item a cluster): the
// parts' O, m and l go to the CTA that writes the rows through distributed shared memory and are joined there.
// Roles (384 threads):
//   warps 0-3, 4-7  softmax of query tile 0 / 1: one thread per query (TMEM lane), 128 scores in
//                   registers, P written back over the scores as bf16; O / l at the end;
//   warp 8          TMA: the query tiles, then K (two 64-dim slabs of k_nope, one of k_pe) and V
//                   (two slabs) of each 128-key tile through a ring of eight 16 KB slabs;
//   warp 9          MMA: S = Q K^T with both operands in shared memory, O += P V with P in tensor
//                   memory, alternating between the query tiles;
//   warp 10         the work items: claims the next one, finds its request and rows (warp 11 idle).
// Tensor memory (512 columns): S / P of tile 0, of tile 1, O of tile 0, of tile 1 (128 each).
// Shared memory: queries 96 KB, ring 128 KB.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace dsa {
namespace {

using namespace attn;

constexpr int kMaxKeys = 1 << 26;                         // an item stays within the limit of a wait (about 2 s)
constexpr int kTileQ = 128, kTileK = 128, kBlockQ = 2 * kTileQ;
constexpr int kSlabBytes = 128 * 128;                     // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kRing = 8;
constexpr int kQSlabs = 3, kKSlabs = 3, kVSlabs = 2;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kWorkWarp = 10;
constexpr int kPreThreads = 384;                          // three warpgroups; warp 11 only fills the third
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;        // 2 x 128 x 208 + 128 x 88 <= 384 x 168 at launch
// Split items: the parts of a row group of 32 queries (a softmax warp's) are joined by one CTA; a part is
// 32 x 128 fp32 outputs, then the rows' maxima (log2 units) and sums.
constexpr int kGroups = 8, kPartBytes = 32 * 512 + 256, kMaxSplit = 4;
static_assert(2 * (kGroups - kGroups / kMaxSplit) * kPartBytes <= (2 * kQSlabs + kRing) * kSlabBytes, "parts sent and received");
constexpr int64_t kGroupBytes = 96 << 20;                 // keys and values of a group of heads (L2: 129 MB)
constexpr uint32_t kColS = 0, kColO = 256;                // + 128 * tile
constexpr size_t kPreSmem = 1024 + size_t(2 * kQSlabs + kRing) * kSlabBytes + 512;
static_assert(kPreSmem <= 232448, "shared-memory budget");

struct Work {
    int b;                   // request; -1: no more work
    int h, qb, q0, nq;       // head, query block, first query row and queries of the request
    int k0, nk;              // first key row and keys (of this CTA's part of the request)
    int diag;                // causal: query i sees the first diag + i + 1 of them
};

struct PreBars {
    uint64_t q_full[2], q_empty[2];      // queries of the tile in place / read by the item's last S, per item
    uint64_t full[kRing], empty[kRing];
    uint64_t s_full[2];      // scores of the tile's next step complete (and with them its previous P V)
    uint64_t p_full[2];      // P written (4 softmax warps)
    uint64_t o_full[2];      // the item's last P V complete
    uint64_t o_free[2];      // O read out (4 softmax warps), per item
    uint64_t work_full[2], work_empty[2];   // a work item published / done with (TMA, MMA and 8 softmax warps)
    uint64_t claim_full;     // answer to the claim of another block
    alignas(16) uint32_t claim[4];
    Work work[2];
    uint64_t joined[8 / 2];  // split items: the parts of a row group arrived (armed + bytes)
    uint32_t tmem_slot;
};
static_assert(sizeof(PreBars) <= 512, "barrier block");

// Asks for the item of a block that has not started; the 16-byte answer is counted on `bar`.
__device__ __forceinline__ void claim_block(uint32_t* answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     ptx::smem_addr(answer)),
                 "r"(ptx::smem_addr(bar))
                 : "memory");
}
// Whether a block was claimed, and which.
__device__ __forceinline__ bool claimed_block(const uint32_t* answer, int& x, int& y) {
    uint32_t ok, bx, by;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%3];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, r;\n\t}"
        : "=r"(ok), "=r"(bx), "=r"(by)
        : "r"(ptx::smem_addr(answer))
        : "memory");
    x = static_cast<int>(bx);
    y = static_cast<int>(by);
    return ok != 0;
}

// Where the last search ended: the chunk of 32 requests and the blocks before it.  Claimed blocks come in
// ascending order, so a search goes on from there; from the start for each would cost a memory latency
// per 32 requests and item.
struct Scan {
    int b0, before;
};

// Block x in the order of requests, the last (longest) query block of each first; false: past the last.
__device__ __forceinline__ bool find_item(const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int B, int T,
                                          int S, int x, int h, int lane, Scan& scan, Work* item, int32_t* err) {
    const bool check = x == 0 && h == 0;                       // this one looks at every request's range
    if (x < scan.before) scan = Scan{0, 0};
    int carry = scan.before;
    bool found = false;
    for (int b0 = scan.b0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        int q0 = 0, nq = 0;
        if (b < B) {
            const int lo = __ldg(cu_q + b), hi = __ldg(cu_q + b + 1);
            q0 = max(0, min(T, lo));
            nq = max(0, min(T, hi) - q0);
            if (check && (lo < 0 || hi > T)) raise_error(err, DSA_DEVERR_INDEX_RANGE);
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
            scan = Scan{b0, carry};
            if (lane == __ffs(hit) - 1) {
                const int lo = __ldg(cu_k + b), hi = __ldg(cu_k + b + 1);
                const int k0 = max(0, min(S, lo));
                if (lo < 0 || hi > S) raise_error(err, DSA_DEVERR_INDEX_RANGE);
                *item = Work{b, h, nb - 1 - (x - (carry + inc - nb)), q0, nq, k0, max(0, min(S, hi) - k0), 0};
                item->diag = item->nk - nq;
            }
            if (!check) break;
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    __syncwarp();
    return found;
}

// Key tiles that the rows of the item's two query tiles see.
struct Tiles {
    int n[2] = {0, 0}, most = 0;
    Tiles() = default;
    __device__ Tiles(const Work& w, int causal) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int first = w.qb * kBlockQ + i * kTileQ;
            const int last = min(w.nq, first + kTileQ) - 1;
            const int seen = last < first ? 0 : (causal ? max(0, min(w.nk, w.diag + last + 1)) : w.nk);
            n[i] = (seen + kTileK - 1) / kTileK;
        }
        most = max(n[0], n[1]);
    }
};

template <int C>
__global__ void __launch_bounds__(kPreThreads, 1)
dense_mla_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap vmap,
                         const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int B, int T, int S, int H,
                         float scale, int causal, int group, uint16_t* __restrict__ out, int64_t out_row, int64_t out_head,
                         float* __restrict__ lse_out, int32_t* err) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    unsigned char* qs = base;                                  // [2 tiles][3 slabs]
    unsigned char* ring = base + 2 * kQSlabs * kSlabBytes;     // [8]
    PreBars& bar = *reinterpret_cast<PreBars*>(ring + kRing * kSlabBytes);

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (warp == kTmaWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bar.q_full[i], 1);
            ptx::mbar_init(&bar.q_empty[i], 1);
            ptx::mbar_init(&bar.s_full[i], 1);
            ptx::mbar_init(&bar.p_full[i], 4);
            ptx::mbar_init(&bar.o_full[i], 1);
            ptx::mbar_init(&bar.o_free[i], 4);
            ptx::mbar_init(&bar.work_full[i], 1);
            ptx::mbar_init(&bar.work_empty[i], 10);
        }
        ptx::mbar_init(&bar.claim_full, 1);
        if constexpr (C > 1)
            for (int g = 0; g < kGroups / C; ++g) {
                ptx::mbar_init(&bar.joined[g], 1);
                ptx::mbar_arrive_expect_tx(&bar.joined[g], (C - 1) * kPartBytes);
            }
        for (int s = 0; s < kRing; ++s) {
            ptx::mbar_init(&bar.full[s], 1);
            ptx::mbar_init(&bar.empty[s], 1);
        }
        ptx::fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&bar.tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();   // a programmatic dependent: what came before is complete
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem_slot);
    // limit of every wait, set anew with every work item (one lasts at most about a second: kMaxKeys)
    uint64_t deadline = ptx::wait_deadline();
    bool timed_out = false, synced = false;               // synced (C > 1): this warp has met the cluster
    // Work item k has been published, or there is no more (whole warp).  `done` gives its slot back; the
    // softmax warps do so at the item's end, which holds the claims one item ahead.
    uint32_t k = 0;
    auto have_work = [&]() -> bool {
        deadline = ptx::wait_deadline();
        if (!ptx::mbar_wait(&bar.work_full[k & 1u], (k >> 1) & 1u, deadline)) timed_out = true;
        timed_out = __any_sync(0xffffffffu, timed_out);
        deadline = ptx::wait_deadline();
        return !timed_out && uniform(bar.work[k & 1u].b) >= 0;
    };
    auto copy_work = [&]() -> Work {
        const Work& x = bar.work[k & 1u];
        return Work{0, uniform(x.h), uniform(x.qb), uniform(x.q0), uniform(x.nq), uniform(x.k0), uniform(x.nk), uniform(x.diag)};
    };
    auto done = [&]() {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar.work_empty[k & 1u]);
        ++k;
    };

    if (warp >= kTmaWarp) {
        set_regs_dec<kOtherRegs>();
        if (warp == kWorkWarp) {
            // ---------------------------------------------------------------- work items
            int x = static_cast<int>(blockIdx.x) / C, y = static_cast<int>(blockIdx.y);
            uint32_t claim_phase = 0;
            Scan scan{0, 0};
            for (uint32_t j = 0;;) {
                deadline = ptx::wait_deadline();
                // the slot's previous item is done with by every warp
                if (j >= 2 && !ptx::mbar_wait(&bar.work_empty[j & 1u], ((j >> 1) & 1u) ^ 1u, deadline)) timed_out = true;
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                // the first item is the CTA's own block; every other one is claimed
                bool found = false;
                for (bool claim = j > 0;; claim = true) {
                    if (claim) {
                        if constexpr (C > 1) break;                  // one item a cluster
                        if (lane == 0) {
                            ptx::fence_proxy_async_smem();           // the answer before has been read
                            ptx::mbar_arrive_expect_tx(&bar.claim_full, 16);
                            claim_block(bar.claim, &bar.claim_full);
                        }
                        if (!ptx::mbar_wait(&bar.claim_full, claim_phase & 1u, deadline)) timed_out = true;
                        ++claim_phase;
                        timed_out = __any_sync(0xffffffffu, timed_out);
                        if (timed_out) break;
                        const bool more = claimed_block(bar.claim, x, y);
                        __syncwarp();
                        if (!more) break;
                    }
                    // the grid's order, x first, as (group of heads, block, head): a prompt's long blocks of many heads
                    // come first, and its last items are short ones (8K prompt x 16 heads: one head after the other
                    // 292 us, so 210)
                    const int blocks = static_cast<int>(gridDim.x) / C, id = y * blocks + x;
                    const int g0 = id / (group * blocks) * group, heads = min(group, H - g0), rem = id - g0 * blocks;
                    found = find_item(cu_q, cu_k, B, T, S, rem / heads, g0 + rem % heads, lane, scan, &bar.work[j & 1u], err);
                    if (found) break;
                }
                if (timed_out) break;
                if constexpr (C > 1) {
                    if (found) {                                     // this CTA's share of the item's key tiles
                        Work w = bar.work[0];
                        const Tiles all(w, causal);
                        const int rank = static_cast<int>(blockIdx.x) % C, from = all.most * rank / C * kTileK;
                        w.nk = max(0, min(w.nk, all.most * (rank + 1) / C * kTileK) - from);
                        w.k0 += from;
                        w.diag -= from;
                        __syncwarp();
                        if (lane == 0) bar.work[0] = w;
                    }
                }
                if (!found && lane == 0) bar.work[j & 1u].b = -1;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.work_full[j & 1u]);
                ++j;
                if (!found) break;
            }
        } else if (warp == kTmaWarp) {
            // ---------------------------------------------------------------- TMA
            uint32_t c = 0, qn[2] = {0, 0};                        // slabs issued; items that used the query tile
            while (have_work()) {
                const Work w = copy_work();
                const Tiles n(w, causal);
                if (lane == 0 && n.most > 0) {
                    auto next = [&]() -> unsigned char* {          // the ring's next slab, once it is free
                        const int s = static_cast<int>(c % kRing);
                        if (!ptx::mbar_wait(&bar.empty[s], ((c / kRing) & 1u) ^ 1u, deadline)) timed_out = true;
                        if (timed_out) return nullptr;
                        ptx::mbar_arrive_expect_tx(&bar.full[s], kSlabBytes);
                        ++c;
                        return ring + s * kSlabBytes;
                    };
                    auto bar_of_last = [&]() { return &bar.full[(c - 1) % kRing]; };
                    auto load_q = [&](int i) {
                        if (n.n[i] == 0 || timed_out) return;
                        if (qn[i] > 0 && !ptx::mbar_wait(&bar.q_empty[i], (qn[i] - 1) & 1u, deadline)) {
                            timed_out = true;
                            return;
                        }
                        ++qn[i];
                        ptx::mbar_arrive_expect_tx(&bar.q_full[i], kQSlabs * kSlabBytes);
                        for (int j = 0; j < kQSlabs; ++j)
                            ptx::tma_load_3d(qs + (i * kQSlabs + j) * kSlabBytes, &qmap, &bar.q_full[i], 64 * j, w.h,
                                             w.q0 + w.qb * kBlockQ + i * kTileQ);
                    };
                    auto load_k = [&](int t) {
                        for (int j = 0; j < kKSlabs && !timed_out; ++j)
                            if (unsigned char* dst = next()) {
                                if (j < 2) ptx::tma_load_3d(dst, &kmap, bar_of_last(), 64 * j, w.h, w.k0 + t * kTileK);
                                else ptx::tma_load_3d(dst, &pmap, bar_of_last(), 0, 0, w.k0 + t * kTileK);
                            }
                    };
                    load_q(0);
                    load_k(0);
                    load_q(1);
                    for (int t = 0; t < n.most && !timed_out; ++t) {
                        const int swap = c % kRing == kRing - 1 ? 1 : 0;   // see issue_pv
                        for (int j = 0; j < kVSlabs && !timed_out; ++j)
                            if (unsigned char* dst = next())
                                ptx::tma_load_3d(dst, &vmap, bar_of_last(), 64 * (j ^ swap), w.h, w.k0 + t * kTileK);
                        if (t + 1 < n.most) load_k(t + 1);
                    }
                }
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                done();
            }
            // copies still in flight land before the CTA may leave (bounded)
            if (lane == 0) {
                for (int i = 0; i < 2; ++i)
                    if (qn[i] > 0 && !ptx::mbar_wait(&bar.q_full[i], (qn[i] - 1) & 1u, ptx::wait_deadline(20000000ull)))
                        timed_out = true;
                for (uint32_t j = c > kRing ? c - kRing : 0; j < c; ++j)
                    if (!ptx::mbar_wait(&bar.full[j % kRing], (j / kRing) & 1u, ptx::wait_deadline(20000000ull)))
                        timed_out = true;
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- MMA
            constexpr uint32_t idesc_qk = ptx::instr_desc(1, 1, kTileQ, kTileK);
            constexpr uint32_t idesc_pv = ptx::instr_desc(1, 1, kTileQ, 128) | (1u << 16);   // B MN-major
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
            // Descriptors differ in their low word only.  What an MMA takes is made uniform right before it issues:
            // the operands are uniform registers, and values that the compiler cannot tell to be the same in
            // all lanes are moved there one by one for each MMA (8 prompts of 128 to 2048: 385 -> 361 us, together
            // with V's swapped halves below, which had been products of half the width).
            const uint64_t q_desc = desc_sw128(q_addr, 16, 1024), k_desc = desc_sw128(ring_addr, 16, 1024);
            const uint64_t v_desc = desc_sw128(ring_addr, kSlabBytes, 1024);
            const uint64_t v_wrap = desc_sw128(ring_addr, (kRing - 1) * kSlabBytes, 1024);
            auto low = [](uint64_t d) { return static_cast<uint32_t>(d); };
            auto with_low = [](uint64_t d, uint32_t lo) { return (d & 0xffffffff00000000ull) | lo; };
            auto slab = [&](uint32_t cc) { return (cc % kRing) * (kSlabBytes / 16); };
            // S_i = Q_i K^T from the slabs at c0; the first user of a key tile waits for each slab in turn;
            // the item's last one gives the queries back
            auto issue_s = [&](int i, uint32_t c0, bool first, bool last) {
#pragma unroll
                for (int j = 0; j < kKSlabs; ++j) {
                    if (first) {
                        wait_slab(c0 + j);
                        __syncwarp();
                        ptx::tc_fence_after_sync();
                    }
                    const uint32_t a = uniform(low(q_desc) + i * (kQSlabs * kSlabBytes / 16) + j * (kSlabBytes / 16));
                    const uint32_t bk = uniform(low(k_desc) + slab(c0 + j)), d = uniform(tmem + kColS + 128 * i);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::umma_f16(d, with_low(q_desc, a + kk * 2), with_low(k_desc, bk + kk * 2), idesc_qk,
                                          (j | kk) != 0 ? 1u : 0u);
                        if (j == kKSlabs - 1) {
                            ptx::umma_commit(&bar.s_full[i]);
                            if (last) ptx::umma_commit(&bar.q_empty[i]);
                        }
                    }
                }
            };
            // O_i += P_i V from the two slabs at c0.  Where the ring wraps between them the halves of V lie
            // swapped: dims 0-63 in the first slab, 64-127 in the last.
            auto issue_pv = [&](int i, uint32_t c0, uint32_t accumulate) {
                const bool wrap = c0 % kRing == kRing - 1;
                const uint32_t bv = uniform(wrap ? low(v_wrap) : low(v_desc) + slab(c0));
                const uint32_t o = uniform(tmem + kColO + 128 * i), p = uniform(tmem + kColS + 128 * i);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kTileK / 16; ++ks)
                        umma_f16_ts(o, p + ks * 8, with_low(v_desc, bv + ks * 128), idesc_pv, ks != 0 ? 1u : accumulate);
                }
            };
            // A step issues P V of its key tile and the scores of the next one.  In an item's last step the next
            // one is the first of the item after it (K of that lies behind the last V in the ring, too), so the
            // tensor cores work while the softmax warps write the output, and a causal item's tile 0, one step
            // shorter, goes on at once.
            Tiles n, nn;                                       // of this item and the next
            int nk = 0, nk_next = 0;
            bool more = false;
            uint32_t c_k = 0;                                  // first slab of the next K
            uint32_t q_phase = 0, p_phase = 0, o_phase = 0, o_used = 0;   // bit i: of the tile's barriers
            auto step = [&](int t, bool over) {
                // ring order: K(0), V(0), K(1), V(1), ...
                const uint32_t c_v = c_k - kVSlabs;
                const int last = t < n.n[1] ? 1 : 0;           // the last tile that uses V(t)
                if (over) {
                    // one item ahead and no further: the one after it is published when the softmax warps are done
                    // with this one, for which they need the products of this step
                    more = have_work();
                    if (more) {
                        const Work w = copy_work();
                        nn = Tiles(w, causal);
                        nk_next = w.nk;
                        done();
                    }
                }
                const bool next_k = over ? more && nn.most > 0 : true;   // K behind this step's V
                bool first_v = true, first_k = true;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t bit = 1u << i;
                    const int ni = i == 0 ? n.n[0] : n.n[1];
                    if (t >= 0 && t < ni) {
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
                        if (t == 0) {                                  // the item before has read its output
                            if ((o_used & bit) != 0u) {
                                wait(&bar.o_free[i], (o_phase >> i) & 1u);
                                o_phase ^= bit;
                            }
                            o_used |= bit;
                        }
                        wait(&bar.p_full[i], (p_phase >> i) & 1u);
                        p_phase ^= bit;
                        __syncwarp();
                        ptx::tc_fence_after_sync();
                        issue_pv(i, c_v, t != 0 ? 1u : 0u);
                        if (i == last) release(c_v, kVSlabs);
                        if (t + 1 == ni && elect_one()) ptx::umma_commit(&bar.o_full[i]);
                        __syncwarp();
                    }
                    // score tiles of the query tile from the next step on
                    const int left = over ? (!more ? 0 : i == 0 ? nn.n[0] : nn.n[1]) : ni - t - 1;
                    if (left > 0) {
                        if (over) {
                            wait(&bar.q_full[i], (q_phase >> i) & 1u);
                            q_phase ^= bit;
                        }
                        issue_s(i, c_k, first_k, left == 1);
                        first_k = false;
                    }
                }
                if (next_k) {
                    release(c_k, kKSlabs);
                    c_k += kKSlabs + kVSlabs;
                }
            };
            for (;;) {
                // the first time there is no item yet, and one that sees no key has no steps: only the first scores
                // of the next
                for (int t = n.most == 0 ? -1 : 0; t < n.most; ++t) {
                    step(t, t + 1 == n.most);
                    if (__any_sync(0xffffffffu, late)) break;
                }
                if (!more || __any_sync(0xffffffffu, late)) break;
                n = nn;
                nk = nk_next;
            }
            if (late) timed_out = true;
        }
    } else {
        set_regs_inc<kSoftmaxRegs>();
        // ---------------------------------------------------------------- softmax, epilogue
        const int i = warp >> 2;                               // query tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + kColS + 128 * i;
        const uint32_t o_addr = tmem + lane_base + kColO + 128 * i;
        const float cs = scale * kLog2e;
        const uint64_t cs2 = f32x2(cs, cs);
        uint32_t qn = 0, sn = 0;                               // the tile's items and steps so far
        while (have_work()) {
            // the item stays in shared memory and is read again for the output: the scores need the registers
            int n, vis, all_see;
            {
                const Work w = copy_work();
                const Tiles tiles(w, causal);
                n = i == 0 ? tiles.n[0] : tiles.n[1];
                const int row0 = w.qb * kBlockQ + i * kTileQ, row = row0 + (warp & 3) * 32 + lane;
                vis = row < w.nq ? (causal ? max(0, min(w.nk, w.diag + row + 1)) : w.nk) : 0;
                // keys that every row of the tile sees: key tiles below need no mask
                all_see = causal ? min(w.nk, w.diag + row0 + 1) : w.nk;
            }
            float m_run = -INFINITY, l_run = 0.0f;
            for (int t = 0; t < n; ++t, ++sn) {
                if (!ptx::mbar_wait(&bar.s_full[i], sn & 1u, deadline)) timed_out = true;
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
                    if (t > 0) {                               // P V (t - 1) has completed: s_full covers it
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
            if (timed_out) break;
            if (n > 0) {
                if (!ptx::mbar_wait(&bar.o_full[i], qn & 1u, deadline)) timed_out = true;
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                ptx::tc_fence_after_sync();
            }
            const Work w = copy_work();
            const int row0 = w.qb * kBlockQ + i * kTileQ, row = row0 + (warp & 3) * 32 + lane;   // query of the request
            float m2 = m_run * cs, l_all = l_run;              // maximum (log2 units) and sum of all parts
            float weight[C];                                   // of this CTA's part and the others'; 0: not counted
            const unsigned char* part = nullptr;               // the others', kPartBytes each
            if constexpr (C > 1) {
                // The row groups are shared out over the cluster; a CTA sends its part of the others' groups through
                // the shared memory that queries, keys and values had, and joins the parts of its own.
                constexpr int kOwn = kGroups / C;
                const int rank = static_cast<int>(blockIdx.x) % C, owner = warp / kOwn, group = warp % kOwn;
                cluster_sync_all();                            // no CTA of the cluster uses it for them any more
                synced = true;
                unsigned char* recv = qs + (kGroups - kOwn) * kPartBytes;
                if (owner != rank) {
                    unsigned char* send = qs + (owner < rank ? warp : warp - kOwn) * kPartBytes;
                    if (n > 0) {
#pragma unroll 1
                        for (int cc = 0; cc < 128; cc += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4*>(send + lane * 512 + (((cc / 4 + e) ^ lane) << 4)) =
                                    make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                        ptx::tc_fence_before_sync();
                    }
                    *reinterpret_cast<float*>(send + 16384 + lane * 4) = m2;
                    *reinterpret_cast<float*>(send + 16512 + lane * 4) = l_run;
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one())
                        bulk_to_peer(map_to_rank(ptx::smem_addr(recv) + (group * (C - 1) + (rank < owner ? rank : rank - 1)) * kPartBytes,
                                                 owner),
                                     ptx::smem_addr(send), kPartBytes, map_to_rank(ptx::smem_addr(&bar.joined[group]), owner));
                    done();
                    continue;
                }
                part = recv + group * (C - 1) * kPartBytes;
                if (!ptx::mbar_wait(&bar.joined[group], 0, deadline)) timed_out = true;
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                float pm[C], pl[C], top = l_run > 0.0f ? m2 : -INFINITY;
                pm[0] = m2;
                pl[0] = l_run;
#pragma unroll
                for (int p = 1; p < C; ++p) {
                    pm[p] = *reinterpret_cast<const float*>(part + (p - 1) * kPartBytes + 16384 + lane * 4);
                    pl[p] = *reinterpret_cast<const float*>(part + (p - 1) * kPartBytes + 16512 + lane * 4);
                    if (pl[p] != 0.0f) top = fmaxf(top, pm[p]);
                }
                if (!(l_run > 0.0f) && l_run != 0.0f) top = fmaxf(top, m2);   // NaN sums count, too
                l_all = 0.0f;
#pragma unroll
                for (int p = 0; p < C; ++p) {
                    weight[p] = pl[p] == 0.0f ? 0.0f : exp2f(pm[p] - top);
                    if (weight[p] != 0.0f) l_all = fmaf(weight[p], pl[p], l_all);
                }
                m2 = top;
            }
            const float inv = l_all == 0.0f ? 0.0f : 1.0f / l_all;
            const bool none = C > 1 ? l_all == 0.0f : n == 0 || vis == 0;   // sees nothing: 0 (O may hold 0 x NaN)
            uint16_t* dst = out + static_cast<int64_t>(w.h) * out_head + (lane & 7) * 8;
            const int rows0 = row0 + (warp & 3) * 32 + (lane >> 3) * 8;   // rows this lane writes: rows0 .. + 7
#pragma unroll 1
            for (int cc = 0; cc < 128; cc += 64) {
                uint32_t v[8][4];                              // the row's 16-byte pieces
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t o[32];
                    if (n > 0) {
                        ptx::tmem_ld_32x32b_x32(o_addr + cc + 32 * hh, o);
                        ptx::tmem_wait_ld();
                    }
                    if constexpr (C > 1) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = weight[0] == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[e]) * weight[0]);
#pragma unroll
                        for (int p = 1; p < C; ++p) {
                            if (weight[p] == 0.0f) continue;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 x = *reinterpret_cast<const float4*>(
                                    part + (p - 1) * kPartBytes + lane * 512 + (((cc / 4 + 8 * hh + e) ^ lane) << 4));
                                o[4 * e] = __float_as_uint(fmaf(weight[p], x.x, __uint_as_float(o[4 * e])));
                                o[4 * e + 1] = __float_as_uint(fmaf(weight[p], x.y, __uint_as_float(o[4 * e + 1])));
                                o[4 * e + 2] = __float_as_uint(fmaf(weight[p], x.z, __uint_as_float(o[4 * e + 2])));
                                o[4 * e + 3] = __float_as_uint(fmaf(weight[p], x.w, __uint_as_float(o[4 * e + 3])));
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[4 * hh + e / 4][e & 3] =
                            none ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                }
                // 8 x 8 transpose of the pieces within each group of 8 lanes, so that 8 lanes write a whole
                // 128-byte line (a thread that writes its own row touches 32 lines per store)
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) {
                    const bool upper = (lane & m) != 0;
#pragma unroll
                    for (int a = 0; a < 8; ++a) {
                        if (a & m) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t mine = upper ? v[a][e] : v[a | m][e];
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, mine, m);
                            if (upper) v[a][e] = got;
                            else v[a | m][e] = got;
                        }
                    }
                }
#pragma unroll
                for (int a = 0; a < 8; ++a)
                    if (rows0 + a < w.nq)
                        *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(w.q0 + rows0 + a) * out_row + cc) =
                            make_uint4(v[a][0], v[a][1], v[a][2], v[a][3]);
            }
            if (n > 0) {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.o_free[i]);
                ++qn;
            }
            if (row < w.nq && lse_out != nullptr)
                lse_out[static_cast<int64_t>(w.q0 + row) * H + w.h] =
                    l_all == 0.0f ? -INFINITY : (m2 + log2f(l_all)) * kLn2;
            done();
        }
    }
    if (timed_out) raise_error(err, DSA_DEVERR_TIMEOUT);
    if constexpr (C > 1) {
        __syncwarp();
        if (!synced) cluster_sync_all();
        cluster_sync_all();                                    // the parts sent have arrived: shared memory may go
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

struct Plan {
    int split;               // CTAs per item
    int group;               // heads whose items are taken longest first
};

// Both from the lengths of an average request, T / B and S / B of the arrays: the lengths themselves are on the
// device.  One long prompt among many short ones is therefore planned like the short ones, and a padded batch like
// its padding.  Splitting an item's keys pays where items are few and of like
// length: a call takes about as many steps of a key tile (1.7 us) as its longest CTA, and an item on a cluster of
// 2 or 4 takes a launch and a join as long as 4 or 8 of them (1000 queries after 15001 keys, CTAs per item 1, 2
// and 4: 8 heads 211, 115 and 66 us; 16 heads 214, 115 and 130; 128 heads 850, 790 and 945).  Items of unlike
// length (a prompt without earlier keys) balance by themselves, the long ones of a group first, unless there are
// fewer than CTAs; a group is as large as the keys and values of its heads stay in L2 (8K prompt, 128 heads: single
// heads 1.66 ms, 22 at a time 1.58, all at once 1.83).  Items of like length go head by head.
Plan make_plan(int64_t T, int64_t S, int64_t B, int64_t H, int64_t blocks, bool causal) {
    const int64_t sms = device_sm_count(), queries = (T + B - 1) / B, keys = std::max<int64_t>(1, (S + B - 1) / B);
    const double longest = static_cast<double>(keys) / kTileK;
    const double mean = longest - (causal ? static_cast<double>(std::min(queries, keys)) / (2 * kTileK) : 0.0);
    const bool alike = mean > 0.75 * longest;
    const int64_t items = (queries + kBlockQ - 1) / kBlockQ * B * H;
    const double alone = alike ? static_cast<double>((items + sms - 1) / sms) * longest
                               : std::max(longest, static_cast<double>(items) * mean / static_cast<double>(sms) + longest / 5);
    int best = 1;
    double least = 0.95 * alone;
    for (int c = 2; c <= kMaxSplit; c *= 2) {
        // clusters at a time; of four, 36 fit the 152 SMs (they do not span groups of SMs)
        const int64_t fit = std::max<int64_t>(1, c == 2 ? sms / 2 : sms / 4 - 2), waves = (blocks * H + fit - 1) / fit;
        if (!alike && waves > 1) continue;
        const double steps = static_cast<double>(waves) * (longest / c + 2 * c);
        if (steps < least) {
            best = c;
            least = steps;
        }
    }
    const int64_t most = std::max<int64_t>(1, kGroupBytes / (keys * 512)), groups = (H + most - 1) / most;
    return Plan{best, alike ? 1 : static_cast<int>((H + groups - 1) / groups)};   // groups of equal size
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
    if (static_cast<int64_t>(T) * H >= 0x7fffffffLL || H > 65535 || S > kMaxKeys) return DSA_ERR_UNSUPPORTED;
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
    // at least the sum of the requests' blocks (ceil(n / 256) <= (n + 255) / 256 each)
    const int64_t blocks = (T + (kBlockQ - 1) * static_cast<int64_t>(std::min(B, T))) / kBlockQ;
    const bool causal = (flags & DSA_CAUSAL) != 0;
    const Plan plan = make_plan(T, S, B, H, blocks, causal);
    const int split = plan.split;
    auto kernel = split == 1 ? dense_mla_prefill_kernel<1> : split == 2 ? dense_mla_prefill_kernel<2> : dense_mla_prefill_kernel<4>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPreSmem)) != cudaSuccess)
        return DSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * split), static_cast<unsigned>(H));
    cfg.blockDim = dim3(kPreThreads);
    cfg.dynamicSmemBytes = kPreSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, qmap, kmap, pmap, vmap, cu_q, cu_k, B, T, S, H, scale, causal ? 1 : 0, plan.group,
                           static_cast<uint16_t*>(out_bf16), out_row_stride, out_head_stride, lse, dev_err) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}
