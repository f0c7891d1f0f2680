// dense_mla_decode.cu -- absorbed latent attention of new tokens over the whole paged latent cache
// (sm_103a).
//
// Follows vllm mla/common.py, MLACommonImpl.forward decode branch (_forward_decode on the absorbed
// query [ql_nope 512, q_pe 64] and the paged latent cache; returns (out, lse)) and merge_attn_states
// (partial results joined by log-sum-exp).
//
// Mathematics: S_j = scale <q, C[j]> over the visible positions, out = softmax(S) C[:, 0:512], in one
// pass with a running maximum m and sum l (P = 2^(c S - c m), c = scale log2 e; m moves only when a
// tile's maximum exceeds it by more than 8 / c).  S, m, l and O are fp32; P is rounded to bf16 for its
// product with C; l sums the unrounded P.  Pieces of a row over disjoint key ranges are normalised and
// joined with weights 2^(lse_i - max lse).
//
// Bound: HBM, 1152 bytes per cached token and request.  A tile of up to 128 query rows (heads x new
// tokens of one request) needs 2176 FLOP per row and key, 70 % of the tensor time that the copy of
// the key takes, and its output accumulator (128 x 512 fp32) fills the tensor memory of an SM.  So a
// row tile is a pipeline over the two CTAs of a cluster: rank 0 forms the scores and the softmax and
// sends P (bf16, 16 KB a page of 64 keys) and the rescaling factors into rank 1's shared memory
// (bulk copies); rank 1 accumulates all 512 output dims and writes them.  Nothing flows back but
// "buffer free", so latencies overlap; the products are 1152 cycles a page in rank 0 and 1024 in rank
// 1, where the copy of a page from HBM takes about 1560.  Both ranks read a page (rank 1 its 512
// value dims), the second time from L2.  Splitting the dims instead, half of the scores' inner
// dimension and of the outputs each, reads every byte once but swaps partial scores every tile: two
// trips over the cluster network in every page's chain, measured at 3200 cycles a page.
//
// Work: the key tiles (128 positions = two pages) of all row tiles in one sequence, cut into equal shares,
// one per cluster (at least kMinShare tiles).  A row tile that lies within one share is written
// directly; the pieces of the others go to the workspace and the combine kernel joins them.
//
// Measured (128 heads, one new token; calls in a captured graph): 64 requests of 4K to 64K 354 us (5.4 TB/s, 80 % of
// the copy rate; 326 us with every load in L2, where the issue of the scores bounds it; 400 one call after the other
// for a second, at the power limit and 1.56 GHz); 32 of 8192 83.6 us (10 of them the combine); 1 of 4096 20.5 us, 1 of
// 64 15.5 us (the chain of one row tile); 8 of about 128K with two rows of 16 heads 173 us (6.0 TB/s, 88 %).
//
// Roles (384 threads), warps 10 and 11 idle:
//   rank 0  warps 0-7  softmax: rows (tensor-memory lanes) 32 (w % 4) .. + 31, page w / 4 of the tile; queries
//                      into tensor memory (value dims) and shared memory (rope dims);
//           warp 8     TMA: 9 chunks of 64 dims a tile, ring of 8;
//           warp 9     MMA: S = Q K^T (N = 128) into two score tiles in turn.
//   rank 1  warps 0-7  O rescaled where a factor is not 1; O / l to the output, 256 dims a warp;
//           warp 8     TMA: the pages' value dims, ring of 4 stages of 256 dims;
//           warp 9     MMA: O += P V, one N = 256 half per stage.
// Tensor memory: rank 0 query chunks (columns 0-255) and score tiles (256-511), rank 1 O (0-511).
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace dsa {
namespace {

using namespace attn;

constexpr int kRows = 128;                                      // query rows of a row tile (MMA M)
constexpr int kKeys = 128;                                      // keys of a tile: two pages
constexpr int kPageChunk = kPage * 128;                         // 8192: 64 keys x 64 dims, 128-byte swizzle
constexpr int kKStageBytes = 2 * kPageChunk, kKStages = 8;      // rank 0: 64 dims of both pages; a tile is 9 stages
constexpr int kVStageBytes = 4 * kPageChunk, kVStages = 4;      // rank 1: 256 dims of one page; a tile is 4 stages
constexpr int kMaxStages = kKStages > kVStages ? kKStages : kVStages;
constexpr int kSBufs = 2, kPBufs = 4;                           // score tiles; P buffers of one page
constexpr int kPvBars = 4;
constexpr int kPBytes = kRows * kPage * 2;                      // 16384: P of a page, K-major, 128-byte swizzle
constexpr int kQRopeBytes = kRows * 128;                        // 16384
constexpr int kPOffset = kKStages * kKStageBytes + kQRopeBytes; // P at the same place in both ranks
constexpr int kDataBytes = kPOffset + kPBufs * kPBytes;
static_assert(kVStages * kVStageBytes <= kPOffset, "rank 1's stages");
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kDecThreads = 384;
constexpr uint32_t kColS = 256;                                 // rank 0: score tiles, behind the query chunks
constexpr int kMaxRequests = 16384;                             // prefix sums of the schedule fit the ring
constexpr int kMinShare = 2;
constexpr int kAhead = 2;                                       // tiles between a page's prefetch and its copy
constexpr size_t kDecSmem = 1024 + size_t(kDataBytes) + 5120;
static_assert(kDecSmem <= 232448, "shared-memory budget");
static_assert(kMaxRequests * 4 <= kDataBytes, "schedule scratch");

struct DecBars {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    // rank 0
    uint64_t q_full;                        // queries in place (8 softmax warps), per row tile
    uint64_t q_read[kKStages];              // the query chunk in the stage has been copied out of it (4 warps)
    uint64_t s_full[kSBufs];                // scores complete; tile_ok written
    uint64_t s_read[kSBufs];                // ... and read (8 warps)
    uint64_t pair[4];                       // both key halves of a row group have written (2 warps)
    uint64_t p_free[kPBufs];                // rank 1's P V that read the buffer is complete
    uint64_t fin_free;                      // rank 1 has read 1 / l (its 8 row warps), per row tile
    // rank 1
    uint64_t p_full[kPBufs];                // P and the factors arrived (armed + bytes)
    uint64_t scaled[2];                     // O rescaled by them (8 row warps), per tile
    uint64_t pv_done[kPvBars];              // P V of the tile complete (more than the tiles the row warps may be ahead)
    uint64_t o_free;                        // O read out (8 row warps), per row tile
    uint64_t fin_full;                      // 1 / l arrived (armed + bytes), per row tile
    uint64_t stage_lent;                    // two ring stages are free for the output, per row tile
    uint64_t stage_back;                    // ... and no longer read (8 row warps)
    uint32_t tmem_slot;
    int page_ok[kMaxStages];                // bit i: page i of the stage is there and its id valid
    int tile_ok[kSBufs];                    // ... of the score tile's pages
    int start[4];                           // first request, first row tile of it, first key tile, tiles of the share
    int first_cluster;                      // cluster that holds the first piece of the first row tile
    float tmax[2][2][kRows];                // rank 0: [tile parity][key half][row]: maximum of the tile
    alignas(16) float alpha[2][kRows];      // the factors of the tile: rank 0's, copied to rank 1
    float fin[kRows];                       // rank 1: 1 / l; -1: nothing visible
};
static_assert(sizeof(DecBars) <= 5120, "barrier block");

struct Batch {
    const int32_t* seq_lens;
    const int32_t* cu_q;
    int B, T, H, max_pages;
    int per;               // query tokens of a row tile: 128 / H
};

// Row tile g of request b: up to 128 / H consecutive query tokens.
struct RowTile {
    int row0, tokens;      // first query token (global row), number of tokens
    int vis0;              // visible keys of the first one (each next one sees one more; may be <= 0)
    int tiles;             // key tiles of the one that sees most
    bool cut;              // visible keys past the block table
};

__device__ __forceinline__ int query_range(const Batch& bt, int b, int& q0) {
    q0 = max(0, min(bt.T, __ldg(bt.cu_q + b)));
    return max(0, min(bt.T, __ldg(bt.cu_q + b + 1)) - q0);
}

// Lengths below 0 count as 0.
__device__ __forceinline__ int seq_len(const Batch& bt, int b) { return max(0, __ldg(bt.seq_lens + b)); }

__device__ __forceinline__ RowTile row_tile(const Batch& bt, int L, int q0, int nq, int g) {
    RowTile t;
    t.row0 = q0 + g * bt.per;
    t.tokens = min(bt.per, nq - g * bt.per);
    t.vis0 = L - nq + g * bt.per + 1;
    const int most = t.vis0 + t.tokens - 1;
    t.cut = most > bt.max_pages * kPage;
    t.tiles = (max(0, min(most, bt.max_pages * kPage)) + kKeys - 1) / kKeys;
    return t;
}

// A share's pieces, one row tile after the other; every role walks them by itself.
struct Walk {
    Batch bt;
    int b, g, q0, nq, L, left;
    RowTile rt;
    int t0, t1;            // key tiles [t0, t1) of the piece (t0 == t1: a row tile that sees nothing)
    bool whole, first;     // the piece is its whole row tile; the share's first piece

    __device__ Walk(const Batch& batch, const int* start) : bt(batch) {
        b = uniform(start[0]);
        g = uniform(start[1]);
        t0 = uniform(start[2]);
        left = uniform(start[3]);
        first = true;
        load_request();
        set_piece();
    }
    __device__ void load_request() {
        nq = uniform(query_range(bt, b, q0));
        q0 = uniform(q0);
        L = uniform(seq_len(bt, b));
    }
    __device__ void set_piece() {
        rt = row_tile(bt, L, q0, nq, g);
        const int n = max(1, rt.tiles);
        const int take = min(n - t0, left);
        whole = take == n;
        left -= take;
        t1 = min(t0 + take, rt.tiles);
    }
    // false: the share is done
    __device__ bool next() {
        if (left <= 0) return false;
        t0 = 0;
        first = false;
        if ((g + 1) * bt.per < nq) {
            ++g;
        } else {
            g = 0;
            do {
                if (++b >= bt.B) return false;
                load_request();
            } while (nq == 0);
        }
        set_piece();
        return true;
    }
};

// Workspace slot of a part: 2 c for the one that starts share c but not its row tile, else 2 c + 1.
__device__ __forceinline__ int64_t piece_slot(int cluster, const Walk& w) {
    return 2 * static_cast<int64_t>(cluster) + ((w.first && w.t0 > 0) ? 0 : 1);
}

// Key tiles of request b over all its row tiles (a row tile that sees nothing counts as one).
__device__ __forceinline__ int request_tiles(const Batch& bt, int b, int32_t* err) {
    int q0;
    const int nq = query_range(bt, b, q0);
    if (err != nullptr && (__ldg(bt.cu_q + b) < 0 || __ldg(bt.cu_q + b + 1) > bt.T)) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    if (nq == 0) return 0;
    const int L = seq_len(bt, b);
    int sum = 0;
    for (int g = 0; g * bt.per < nq; ++g) {
        const RowTile t = row_tile(bt, L, q0, nq, g);
        if (t.cut && err != nullptr) raise_error(err, DSA_DEVERR_INDEX_RANGE);
        sum += max(1, t.tiles);
    }
    return sum;
}

// The share of cluster c: sums of all requests in `sums` (shared), then one warp finds the start.
__device__ __forceinline__ void find_share(const Batch& bt, int c, int clusters, int* sums, DecBars& bar, int32_t* err) {
    for (int b = threadIdx.x; b < bt.B; b += kDecThreads) sums[b] = request_tiles(bt, b, c == 0 ? err : nullptr);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int total = 0;
        for (int b = lane; b < bt.B; b += 32) total += sums[b];
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
        const int share = max((total + clusters - 1) / clusters, kMinShare);
        const int64_t w0 = static_cast<int64_t>(c) * share;
        if (lane == 0) {
            bar.start[3] = w0 < total ? static_cast<int>(min(static_cast<int64_t>(share), total - w0)) : 0;
        }
        if (w0 < total) {
            int carry = 0;
            for (int b0 = 0; b0 < bt.B; b0 += 32) {
                const int b = b0 + lane;
                int inc = b < bt.B ? sums[b] : 0;
                const int own = inc;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += o;
                }
                const uint32_t hit = __ballot_sync(0xffffffffu, w0 < carry + inc);
                if (hit != 0u) {
                    if (lane == __ffs(hit) - 1) {
                        int at = carry + inc - own;            // tiles before the request
                        int q0;
                        const int nq = query_range(bt, b, q0);
                        const int L = seq_len(bt, b);
                        int g = 0;
                        for (;; ++g) {
                            const int n = max(1, row_tile(bt, L, q0, nq, g).tiles);
                            if (w0 < at + n) break;
                            at += n;
                        }
                        bar.start[0] = b;
                        bar.start[1] = g;
                        bar.start[2] = static_cast<int>(w0 - at);
                        bar.first_cluster = at / share;
                    }
                    break;
                }
                carry += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// 4-byte store into another CTA's shared memory, counted as transaction bytes on that CTA's mbarrier
// (the receiver's wait on it orders the data).
__device__ __forceinline__ void st_async_f32(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}
// Tile of shared memory into global memory by TMA, and the waits of the thread that issued it: all but the
// last N groups have read their source; everything is written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(ptx::smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Arrive on a barrier of the peer without ordering anything before it: used for buffers this thread has
// only read (the values are in registers).  A release at cluster scope costs about 2000 cycles here.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive on the barrier at this offset in rank 0 once the MMAs issued so far have completed.
__device__ __forceinline__ void umma_commit_rank0(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_addr(bar)),
        "h"(static_cast<uint16_t>(1))
        : "memory");
}

// What a cluster leaves for the combine kernel: the split row tile whose last piece it computed.
struct Meta {
    int64_t out_row;       // first output row (token * H)
    int rows;              // its rows; 0: none
    int first_cluster;
};

__global__ void __launch_bounds__(kDecThreads, 1) __cluster_dims__(2, 1, 1)
dense_mla_decode_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                        const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap pmap,
                        const uint16_t* __restrict__ kv, int num_pages,
                        const int32_t* __restrict__ block_table, Batch bt, float scale, uint16_t* __restrict__ out,
                        float* __restrict__ lse_out, float* __restrict__ part_lse, Meta* __restrict__ meta, int slot_rows,
                        int32_t* err) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    unsigned char* ring = base;                                                   // both ranks: key / value stages
    unsigned char* qrope = base + kKStages * kKStageBytes;                        // rank 0: [128 rows][64 dims]
    unsigned char* ps = base + kPOffset;                                          // [4 pages][128 rows][64 keys]
    DecBars& bar = *reinterpret_cast<DecBars*>(base + kDataBytes);

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(&bar.kv_full[s], 1);
            ptx::mbar_init(&bar.kv_empty[s], 1);
        }
        ptx::mbar_init(&bar.q_full, 8);
        for (int s = 0; s < kKStages; ++s) ptx::mbar_init(&bar.q_read[s], 4);
        for (int i = 0; i < kSBufs; ++i) {
            ptx::mbar_init(&bar.s_full[i], 2);
            ptx::mbar_init(&bar.s_read[i], 8);
        }
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&bar.pair[i], 2);
        for (int i = 0; i < kPBufs; ++i) {
            ptx::mbar_init(&bar.p_free[i], 1);
            ptx::mbar_init(&bar.p_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&bar.scaled[i], 8);
        for (int i = 0; i < kPvBars; ++i) ptx::mbar_init(&bar.pv_done[i], 1);
        ptx::mbar_init(&bar.o_free, 8);
        ptx::mbar_init(&bar.fin_full, 1);
        ptx::mbar_init(&bar.stage_lent, 1);
        ptx::mbar_init(&bar.stage_back, 8);
        ptx::mbar_init(&bar.fin_free, 8);
        ptx::fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&bar.tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();             // a programmatic dependent: what came before is complete
    find_share(bt, cluster, clusters, reinterpret_cast<int*>(ring), bar, rank == 0 ? err : nullptr);
    ptx::fence_proxy_async_smem();   // the schedule's scratch lies where copies will land
    ptx::tc_fence_before_sync();
    cluster_sync_all();              // both CTAs' barriers exist before the peer signals or writes into them
    ptx::tc_fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem_slot);
    // limit of every wait, set anew every 256 tiles: a wait lasts a tile or so, the kernel may run for seconds
    uint64_t deadline = ptx::wait_deadline();
    bool timed_out = false;
    const bool work = uniform(bar.start[3]) > 0;
    const uint32_t ring_addr = ptx::smem_addr(ring);
    if (threadIdx.x == 0 && rank == 1) meta[cluster].rows = 0;

    if (work && warp == kTmaWarp) {
        // ---------------------------------------------------------------- TMA (both ranks)
        const uint32_t stages = rank == 0 ? kKStages : kVStages;
        Walk w(bt, bar.start);
        uint32_t s = 0, ph = 0, used = 0;                            // stage, its phase, stages used so far
        auto stage = [&]() {                                         // the next stage is free (whole warp)
            if (!ptx::mbar_wait(&bar.kv_empty[s], ph ^ 1u, deadline)) timed_out = true;
            timed_out = __any_sync(0xffffffffu, timed_out);
            return !timed_out;
        };
        auto advance = [&]() {
            __syncwarp();
            ++used;
            if (++s == stages) {
                s = 0;
                ph ^= 1u;
            }
        };
        do {
            // the row tile's queries, 64 dims a stage (rows past its last one are other tokens', or zeros)
            if (rank == 0 && w.t0 < w.t1)
                for (int c = 0; c < 9 && stage(); ++c) {
                    if (elect_one()) {
                        ptx::mbar_arrive_expect_tx(&bar.kv_full[s], kKStageBytes);
                        ptx::tma_load_3d(ring + s * kKStageBytes, &qmap, &bar.kv_full[s], c * 64, 0, w.rt.row0 * bt.H);
                    }
                    advance();
                }
            const int most = w.rt.vis0 + w.rt.tokens - 1;            // visible keys of the token that sees most
            auto load_pages = [&](int t) {                           // page ids of 16 tiles from t on
                const int at = 2 * t + lane;
                const bool needed = at < 2 * w.t1 && at * kPage < most && at < bt.max_pages;
                return needed ? __ldg(block_table + static_cast<int64_t>(w.b) * bt.max_pages + at) : -1;
            };
            int page = -1, page_next = load_pages(w.t0);
            for (int t = w.t0; t < w.t1 && !timed_out; ++t) {
                const int tb = (t - w.t0) & 15;
                if (tb == 0) {
                    deadline = ptx::wait_deadline();
                    page = page_next;
                    page_next = load_pages(t + 16);
                }
                if (rank == 1 && t + kAhead < w.t1) {
                    // the pages kAhead tiles further into L2: rank 0's ring holds less than the latency of HBM times
                    // its rate (418 -> 393 us on 64 requests of 4K to 64K; from rank 0, or further ahead, slower)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int src = 2 * (tb + kAhead) + i;
                        const int near = __shfl_sync(0xffffffffu, page, src & 31), far = __shfl_sync(0xffffffffu, page_next, src & 31);
                        const int pg = src < 32 ? near : far;
                        if (pg >= 0 && pg < num_pages) {
                            const unsigned char* p = reinterpret_cast<const unsigned char*>(kv + static_cast<int64_t>(pg) * (kPage * kLatentDim));
#pragma unroll
                            for (int j = 0; j < kPage * kLatentDim * 2 / 4096; ++j) prefetch_line(p + (j * 32 + lane) * 128);
                        }
                    }
                }
                int row[2], ok = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pg = __shfl_sync(0xffffffffu, page, 2 * tb + i);
                    const bool needed = (2 * t + i) * kPage < most && 2 * t + i < bt.max_pages;
                    const bool there = needed && pg >= 0 && pg < num_pages;
                    // a page that is not there: a box past the end reads zeros, and rank 0 masks its keys
                    row[i] = (there ? pg : num_pages) * kPage;
                    ok |= there ? 1 << i : 0;
                    if (needed && !there && lane == 0 && rank == 0) raise_error(err, DSA_DEVERR_PAGE_RANGE);
                }
                if (rank == 0) {
                    for (int c = 0; c < 9 && stage(); ++c) {
                        if (elect_one()) {
                            bar.page_ok[s] = ok;
                            ptx::mbar_arrive_expect_tx(&bar.kv_full[s], kKStageBytes);
                            ptx::tma_load_3d(ring + s * kKStageBytes, &kvmap, &bar.kv_full[s], c * 64, 0, row[0]);
                            ptx::tma_load_3d(ring + s * kKStageBytes + kPageChunk, &kvmap, &bar.kv_full[s], c * 64, 0, row[1]);
                        }
                        advance();
                    }
                } else {
                    for (int i = 0; i < 4 && stage(); ++i) {         // page i / 2, value dims 256 (i % 2) .. + 255
                        if (elect_one()) {
                            ptx::mbar_arrive_expect_tx(&bar.kv_full[s], kVStageBytes);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                ptx::tma_load_3d(ring + s * kVStageBytes + j * kPageChunk, &kvmap, &bar.kv_full[s],
                                                 (i & 1) * 256 + j * 64, 0, row[i >> 1]);
                        }
                        advance();
                    }
                }
            }
            // rank 1: two stages for the row tile's output
            if (rank == 1 && w.t0 < w.t1 && !timed_out) {
                for (int i = 0; i < 2 && stage(); ++i) {
                    if (elect_one()) {
                        ptx::mbar_arrive(&bar.kv_full[s]);           // nothing to copy: the stage's phase passes
                        if (i == 1) ptx::mbar_arrive(&bar.stage_lent);
                    }
                    advance();
                }
            }
        } while (!timed_out && w.next());
        // copies still in flight land before the CTA may leave (bounded)
        for (uint32_t j = used > stages ? used - stages : 0; j < used; ++j)
            if (!ptx::mbar_wait(&bar.kv_full[j % stages], (j / stages) & 1u, ptx::wait_deadline(20000000ull))) timed_out = true;
    } else if (work && warp == kMmaWarp && rank == 0) {
        // ---------------------------------------------------------------- MMA: S = Q K^T
        constexpr uint32_t idesc = ptx::instr_desc(1, 1, kRows, kKeys);
        const uint64_t k_desc = desc_sw128(ring_addr, 16, 1024), qr_desc = desc_sw128(ptx::smem_addr(qrope), 16, 1024);
        // a wait that ran out only marks the step; the warp leaves at its end
        bool late = false;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) late = true;
        };
        Walk w(bt, bar.start);
        uint32_t u = 0, seg = 0, s = 0, ph = 0, q_phase = 0;          // q_phase: bit s, the phase of q_read[s]
        do {
            if (w.t0 >= w.t1) continue;
            for (int c = 0; c < 9; ++c) {
                wait(&bar.q_read[s], (q_phase >> s) & 1u);
                q_phase ^= 1u << s;
                __syncwarp();
                if (elect_one()) ptx::mbar_arrive(&bar.kv_empty[s]);
                __syncwarp();
                if (++s == kKStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            wait(&bar.q_full, seg & 1u);
            ++seg;
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                const uint32_t sb = u % kSBufs;
                if (u >= kSBufs) wait(&bar.s_read[sb], ((u / kSBufs) & 1u) ^ 1u);
                const uint32_t d = tmem + kColS + sb * kKeys;
#pragma unroll
                for (int c = 0; c < 9; ++c) {
                    wait(&bar.kv_full[s], ph);
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t so = k_desc + s * (kKStageBytes / 16);
                        if (c == 0) {
                            bar.tile_ok[sb] = bar.page_ok[s];
                            ptx::mbar_arrive(&bar.s_full[sb]);       // orders tile_ok for the softmax
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (c < 8) umma_f16_ts(d, tmem + c * 32 + kk * 8, so + kk * 2, idesc, (c | kk) != 0 ? 1u : 0u);
                            else ptx::umma_f16(d, qr_desc + kk * 2, so + kk * 2, idesc, 1u);
                        }
                        ptx::umma_commit(&bar.kv_empty[s]);
                        if (c == 8) ptx::umma_commit(&bar.s_full[sb]);
                    }
                    __syncwarp();
                    if (++s == kKStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (__any_sync(0xffffffffu, late)) break;
            }
        } while (!__any_sync(0xffffffffu, late) && w.next());
        if (late) timed_out = true;
    } else if (work && warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA: O += P V
        constexpr uint32_t idesc = ptx::instr_desc(1, 1, kRows, 256) | (1u << 16);   // B MN-major
        const uint64_t v_desc = desc_sw128(ring_addr, kPageChunk, 1024), p_desc = desc_sw128(ptx::smem_addr(ps), 16, 1024);
        bool late = false;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) late = true;
        };
        Walk w(bt, bar.start);
        uint32_t u = 0, seg = 0, s = 0, ph = 0;
        do {
            if (w.t0 >= w.t1) continue;
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
#pragma unroll
                for (int i = 0; i < 4; ++i) {                        // page i / 2, value dims 256 (i % 2) .. + 255
                    const uint32_t pb = 2 * (u & 1u) + (i >> 1);
                    wait(&bar.kv_full[s], ph);
                    const int valid = w.rt.vis0 + w.rt.tokens - 1 - t * kKeys - (i >> 1) * kPage;
                    if (valid > 0 && valid < kPage) {
                        // rows past the last visible position may hold anything: their P is 0, but 0 times NaN
                        // or infinity is not (a page without visible rows was filled with zeros)
                        __syncwarp();
                        unsigned char* st = ring + s * kVStageBytes;
                        for (int e = lane; e < (kPage - valid) * 8; e += 32)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<uint4*>(st + j * kPageChunk + (valid + (e >> 3)) * 128 + (e & 7) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        ptx::fence_proxy_async_smem();
                    }
                    if ((i & 1) == 0) wait(&bar.p_full[pb], (u >> 1) & 1u);
                    if (i == 0) {
                        if (t == w.t0 && seg > 0) wait(&bar.o_free, (seg - 1) & 1u);
                        wait(&bar.scaled[u & 1], (u >> 1) & 1u);
                    }
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t vb = v_desc + s * (kVStageBytes / 16);
                        const uint64_t pd = p_desc + pb * (kPBytes / 16);
#pragma unroll
                        for (int ks = 0; ks < kPage / 16; ++ks)
                            ptx::umma_f16(tmem + (i & 1) * 256, pd + ks * 2, vb + ks * 128, idesc,
                                          (t > w.t0 || i >= 2 || ks != 0) ? 1u : 0u);
                        ptx::umma_commit(&bar.kv_empty[s]);
                        if ((i & 1) == 1) umma_commit_rank0(&bar.p_free[pb]);
                        if (i == 3) ptx::umma_commit(&bar.pv_done[u % kPvBars]);
                    }
                    __syncwarp();
                    if (++s == kVStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (__any_sync(0xffffffffu, late)) break;
            }
            wait(&bar.stage_back, seg & 1u);
            for (int i = 0; i < 2; ++i) {
                __syncwarp();
                if (elect_one()) ptx::mbar_arrive(&bar.kv_empty[s]);
                if (++s == kVStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            ++seg;
        } while (!__any_sync(0xffffffffu, late) && w.next());
        if (late) timed_out = true;
    } else if (work && warp < kTmaWarp && rank == 0) {
        // ---------------------------------------------------------------- softmax (rank 0)
        const int quad = warp & 3, kh = warp >> 2;
        const int row = quad * 32 + lane;                            // query row of the row tile = tensor-memory lane
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const float cs = scale * kLog2e;
        const uint64_t cs2 = f32x2(cs, cs);
        const int token = row / bt.H;
        const uint32_t p_row = row * 128, p_swz = row & 7;           // the row's place in a P buffer
        // this warp's 32 rows of a P buffer, and their factors, here and in rank 1
        const uint32_t p_here = ptx::smem_addr(ps) + quad * 4096, p_there = map_to_rank(p_here, 1);
        const uint32_t a_here = ptx::smem_addr(&bar.alpha[0][quad * 32]), a_there = map_to_rank(a_here, 1);
        const uint32_t full_there = map_to_rank(ptx::smem_addr(&bar.p_full[0]), 1);
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) timed_out = true;
        };
        uint32_t u = 0, seg = 0, meets = 0, used = 0;                // meets: uses of the pair barrier; used: ring stages
        Walk w(bt, bar.start);
        do {
            const int live = w.rt.tokens * bt.H;
            const bool quad_live = quad * 32 < live;
            // Rows behind the last one are other requests' queries, stale P and its products: nothing reads what comes
            // of them, but zeros there let the tensor cores idle, and a long call runs at the power limit (8 requests of
            // about 128K with two rows of 16 heads, one call after the other: 200 -> 178 us at 1.47 -> 1.74 GHz)
            const bool row_live = row < live;
            const int vis = row_live ? min(w.rt.vis0 + token, bt.max_pages * kPage) : 0;
            float m_run = -INFINITY, l_run = 0.0f;
            if (w.t0 < w.t1) {
                // the row tile's queries out of the ring: value chunks into tensor memory, the rope chunk into its
                // place; even chunks by the warps of page 0, odd ones by those of page 1.  (The score MMAs
                // before are complete: their s_full has been waited for.  Warps without live rows have not passed a
                // fence since, and the stores to come may not move ahead of that wait.)
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < 9; ++c) {
                    const uint32_t st = used % kKStages;
                    if ((c & 1) == kh) {
                        wait(&bar.kv_full[st], (used / kKStages) & 1u);
                        const unsigned char* src = ring + st * kKStageBytes + p_row;
                        if (c < 8) {
                            uint32_t v[32];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint4 r = *reinterpret_cast<const uint4*>(src + ((i ^ p_swz) << 4));
                                v[4 * i] = row_live ? r.x : 0u;
                                v[4 * i + 1] = row_live ? r.y : 0u;
                                v[4 * i + 2] = row_live ? r.z : 0u;
                                v[4 * i + 3] = row_live ? r.w : 0u;
                            }
                            __syncwarp();
                            tmem_st_x32(tmem + lane_base + c * 32, v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)              // the same swizzle in both places
                                *reinterpret_cast<uint4*>(qrope + p_row + 16 * i) =
                                    row_live ? *reinterpret_cast<const uint4*>(src + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
                            ptx::fence_proxy_async_smem();
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&bar.q_read[st]);
                    }
                    ++used;
                }
                tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.q_full);
            }
            used += 9u * static_cast<uint32_t>(max(0, w.t1 - w.t0));
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                const uint32_t sb = u % kSBufs, pb = 2 * (u & 1u) + kh;
                wait(&bar.s_full[sb], (u / kSBufs) & 1u);
                if (quad_live) {
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    uint32_t v[2][32];
                    const uint32_t sa = tmem + lane_base + kColS + sb * kKeys + kh * kPage;
                    ptx::tmem_ld_32x32b_x32(sa, v[0]);
                    ptx::tmem_ld_32x32b_x32(sa + 32, v[1]);
                    const int lim = ((bar.tile_ok[sb] >> kh) & 1) ? vis - t * kKeys - kh * kPage : 0;
                    ptx::tmem_wait_ld();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar.s_read[sb]);
                    if (lim < kPage) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e >= lim) v[e >> 5][e & 31] = 0xff800000u;   // -inf
                    }
                    float mx4[4];
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const float x = __uint_as_float(v[e >> 5][e & 31]);
                        mx4[e & 3] = e < 4 ? x : fmaxf(mx4[e & 3], x);
                    }
                    float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                    // the tile's maximum over both pages (values double-buffered by tile parity)
                    bar.tmax[u & 1][kh][row] = mx;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar.pair[quad]);
                    wait(&bar.pair[quad], meets & 1u);
                    ++meets;
                    mx = fmaxf(mx, bar.tmax[u & 1][kh ^ 1][row]);
                    const bool grow = (mx - m_run) * cs > kRescaleThreshold || (m_run == -INFINITY && mx > -INFINITY);
                    float alpha = 1.0f;
                    if (grow) {
                        alpha = m_run == -INFINITY ? 0.0f : exp2f((m_run - mx) * cs);
                        m_run = mx;
                        l_run *= alpha;
                    }
                    const float neg = m_run == -INFINITY ? 0.0f : -m_run * cs;
                    const uint64_t neg2 = f32x2(neg, neg);
                    uint64_t sum2 = f32x2(0.0f, 0.0f);
                    if (u >= 2) wait(&bar.p_free[pb], ((u >> 1) & 1u) ^ 1u);
                    unsigned char* prow = ps + pb * kPBytes + p_row;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = 8 * i + 2 * e;
                            float a, b;
                            unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(v[k >> 5][k & 31]), __uint_as_float(v[k >> 5][(k & 31) + 1])),
                                                   cs2, neg2), a, b);
                            a = fast_exp2(a);
                            b = fast_exp2(b);
                            sum2 = add_f32x2(sum2, f32x2(a, b));
                            pk[e] = pack_bf16x2(a, b);
                        }
                        *reinterpret_cast<uint4*>(prow + ((i ^ p_swz) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    if (kh == 0) bar.alpha[u & 1][row] = alpha;
                    // one bulk copy a warp: 16-byte st.async stores of the same bytes took about 1000 cycles a page
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) {
                        bulk_to_peer(p_there + pb * kPBytes, p_here + pb * kPBytes, 4096, full_there + pb * 8);
                        if (kh == 0) bulk_to_peer(a_there + (u & 1u) * (kRows * 4), a_here + (u & 1u) * (kRows * 4), 128, full_there + pb * 8);
                    }
                    __syncwarp();
                    float a, b;
                    unpack_f32x2(sum2, a, b);
                    l_run += a + b;
                } else if (lane == 0) {
                    ptx::mbar_arrive(&bar.s_read[sb]);
                }
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
            }
            if (timed_out) break;
            // ---- 1 / l to rank 1; the log-sum-exp (log2 units for a part)
            if (quad_live) {
                float l_tot = 0.0f;
                if (w.t0 < w.t1) {
                    bar.tmax[u & 1][kh][row] = l_run;                // the buffer of the tile before the last: read by both
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar.pair[quad]);
                    wait(&bar.pair[quad], meets & 1u);
                    ++meets;
                    l_tot = l_run + bar.tmax[u & 1][kh ^ 1][row];
                    // the next row tile's first maximum goes to the same buffer: only after both have read
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar.pair[quad]);
                    wait(&bar.pair[quad], meets & 1u);
                    ++meets;
                    if (seg > 0) wait(&bar.fin_free, (seg - 1) & 1u);
                    if (kh == 0)
                        st_async_f32(map_to_rank(ptx::smem_addr(&bar.fin[row]), 1), l_tot == 0.0f ? -1.0f : 1.0f / l_tot,
                                     map_to_rank(ptx::smem_addr(&bar.fin_full), 1));
                }
                if (kh == 0 && row < live) {
                    const float lse2 = l_tot == 0.0f ? -INFINITY : m_run * cs + log2f(l_tot);
                    if (!w.whole) part_lse[piece_slot(cluster, w) * slot_rows + row] = lse2;
                    else if (lse_out != nullptr) lse_out[static_cast<int64_t>(w.rt.row0) * bt.H + row] = lse2 * kLn2;
                }
            }
            if (w.t0 < w.t1) ++seg;
        } while (w.next());
        // rank 1's last signals land here before this CTA may finish
        for (uint32_t j = 2 * u > kPBufs ? 2 * u - kPBufs : 0; j < 2 * u && !timed_out; ++j)
            wait(&bar.p_free[j % kPBufs], (j / kPBufs) & 1u);
    } else if (work && warp < kTmaWarp) {
        // ---------------------------------------------------------------- rescaling, output (rank 1)
        const int quad = warp & 3, dh = warp >> 2;                   // rows 32 quad .. + 31, output dims 256 dh .. + 255
        const int row = quad * 32 + lane;
        const uint32_t o_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + dh * 256;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) timed_out = true;
        };
        uint32_t u = 0, seg = 0, used = 0;                           // used: ring stages before this row tile
        uint32_t clean = 0;                                          // bit i: this row group's P is zero in buffers 2 i and 2 i + 1
        Walk w(bt, bar.start);
        do {
            const int live = w.rt.tokens * bt.H;
            const bool quad_live = quad * 32 < live, has_tiles = w.t0 < w.t1;
            const uint32_t quads = static_cast<uint32_t>((live + 31) / 32);
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                const uint32_t pb = 2 * (u & 1u), pph = (u >> 1) & 1u;
                if (threadIdx.x == 0) {
                    // the second buffer's previous phase is over once its P V is: this warp has not waited for it
                    if (u >= 2) wait(&bar.p_full[pb + 1], pph ^ 1u);
                    ptx::mbar_arrive_expect_tx(&bar.p_full[pb], quads * (kPBytes / 4 + 32 * 4));
                    ptx::mbar_arrive_expect_tx(&bar.p_full[pb + 1], quads * (kPBytes / 4));
                }
                __syncwarp();
                wait(&bar.p_full[pb], pph);
                if (quad_live) {
                    clean &= ~(1u << (u & 1u));
                } else if (((clean >> (u & 1u)) & 1u) == 0u) {
                    // no P comes for these rows.  Only this tile's buffers: rank 0 writes into them again when its
                    // products are complete, into the others it may have sent the next row tile's already
                    clean |= 1u << (u & 1u);
                    for (int e = lane; e < 256; e += 32)
                        *reinterpret_cast<uint4*>(ps + (pb + dh) * kPBytes + quad * 4096 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                    ptx::fence_proxy_async_smem();
                }
                if (quad_live && t > w.t0) {
                    const float alpha = bar.alpha[u & 1][row];
                    if (__any_sync(0xffffffffu, alpha != 1.0f)) {
                        wait(&bar.pv_done[(u - 1) % kPvBars], ((u - 1) / kPvBars) & 1u);
                        __syncwarp();
                        ptx::tc_fence_after_sync();
#pragma unroll 1
                        for (int cc = 0; cc < 256; cc += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st_x32(o_addr + cc, o);
                        }
                        tmem_wait_st();
                        ptx::tc_fence_before_sync();
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.scaled[u & 1]);
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
            }
            if (timed_out) break;
            float inv = -1.0f;                                       // nothing visible: O may hold 0 x NaN
            uint32_t hidden = 0xffffffffu;                           // bit l: row of lane l, nothing visible
            if (has_tiles) {
                if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(&bar.fin_full, quads * 128);
                wait(&bar.fin_full, seg & 1u);
                inv = bar.fin[row];
                // the arrive orders nothing: the ballot, which takes every lane's value, comes before it, so all are read
                // when rank 0 learns that it may write the next ones
                hidden = __ballot_sync(0xffffffffu, inv < 0.0f);
                __syncwarp();
                if (lane == 0) arrive_remote(map_to_rank(ptx::smem_addr(&bar.fin_free), 0));
                wait(&bar.pv_done[(u - 1) % kPvBars], ((u - 1) / kPvBars) & 1u);
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                ptx::tc_fence_after_sync();
            }
            if (has_tiles) {
                // 128 bytes of each row at a time into 4 KB of a lent stage (128-byte swizzle) and out by TMA, 16 rows
                // a copy (rows come in multiples of 16), one buffer filling while the other leaves.  Stores by
                // threads, whole lines each, went out at 32 bytes a cycle, 4100 (parts: 8200) cycles a row tile
                // (512 requests of 512 keys 124 -> 116 us, one of 4096 22.3 -> 21.1 us).
                used += 4u * static_cast<uint32_t>(w.t1 - w.t0);
                wait(&bar.stage_lent, seg & 1u);
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                const int width = w.whole ? 64 : 32;                 // dims of 128 bytes
                const int64_t row0 = w.whole ? static_cast<int64_t>(w.rt.row0) * bt.H : piece_slot(cluster, w) * slot_rows;
                const int swz = lane & 7;
                int buf = 0;
#pragma unroll 1
                for (int cc = 0; quad_live && cc < 256; cc += width, buf ^= 1) {
                    uint32_t o[32];                                  // the row's 128 bytes
                    ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                    if (w.whole) {
                        uint32_t x[32];
                        ptx::tmem_ld_32x32b_x32(o_addr + cc + 32, x);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[16 + e] = pack_bf16x2(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
                    } else {
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
                    }
                    unsigned char* st = ring + ((used + buf) % kVStages) * kVStageBytes + warp * 4096;
                    if (lane == 0) bulk_wait_read<1>();              // the buffer's previous copies have read it
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(st + lane * 128 + ((i ^ swz) << 4)) =
                            (hidden >> lane) & 1u ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (quad * 32 + 16 * h < live)
                                tma_store_3d(w.whole ? &omap : &pmap, st + h * 2048, dh * 256 + cc, 0,
                                             static_cast<int>(row0) + quad * 32 + 16 * h);
                        bulk_commit();
                    }
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(&bar.o_free);
                    bulk_wait_read<0>();
                    ptx::mbar_arrive(&bar.stage_back);
                }
                used += 2;
                ++seg;
            } else if (quad_live) {                                  // sees nothing: zeros
                for (int r = quad * 32; r < min(live, quad * 32 + 32); ++r)
                    *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(w.rt.row0) * bt.H + r) * kValueDim + dh * 256 + lane * 8) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            // the last piece of a split row tile: the combine kernel finds it here
            if (threadIdx.x == 0 && w.first && w.t0 > 0 && w.t1 == w.rt.tiles)
                meta[cluster] = Meta{static_cast<int64_t>(w.rt.row0) * bt.H, live, bar.first_cluster};
        } while (w.next());
        if (lane == 0) bulk_wait_all();                              // written before the CTA leaves
    }
    if (timed_out) raise_error(err, DSA_DEVERR_TIMEOUT);
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
    cluster_sync_all();   // neither CTA leaves while its peer may still signal or write into it
}

// Joins the pieces of the split row tiles.  The first piece lies in slot 2 c0 + 1, the following ones in slots
// 2 (c0 + 1), .., 2 c.  Bound by the latency of its loads: a task is 128 dims of an output row, four pieces at a
// time, when there are few rows, and a whole row, two pieces at a time, when there are many (512 requests of 512
// keys 116 -> 112 us, 32 of 8192 84.1 -> 83.0; without this kernel 98 and 73).
constexpr int kCombThreads = 256;
constexpr int kCombBlocks = 4;     // per SM (32 requests of 8K: 1 block an SM 33 us of the call, 2 to 8 about 15)

// V x 128 dims from d0 on of one row, P pieces at a time: their sums and values are loaded together.
template <int V, int P>
__device__ __forceinline__ void join_row(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                         const Meta& m, int c, int slot_rows, int row, int d0, int lane,
                                         uint16_t* __restrict__ out, float* __restrict__ lse_out) {
    const int n = c - m.first_cluster + 1;
    auto slot_of = [&](int j) {
        return static_cast<int64_t>(j == 0 ? 2 * m.first_cluster + 1 : 2 * (m.first_cluster + j)) * slot_rows + row;
    };
    float m_run = -INFINITY, tot = 0.0f;
    float4 acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j0 = 0; j0 < n; j0 += P) {
        float l[P];
        float4 o[P][V];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t s = slot_of(min(j0 + i, n - 1));
            l[i] = j0 + i < n ? part_lse[s] : -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) o[i][v] = *reinterpret_cast<const float4*>(part_o + s * kValueDim + d0 + v * 128 + lane * 4);
        }
        float top = m_run;
#pragma unroll
        for (int i = 0; i < P; ++i) top = fmaxf(top, l[i]);
        const float ref = top == -INFINITY ? 0.0f : top;                 // nothing visible so far: weights 0
        const float f = exp2f(m_run - ref);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = make_float4(acc[v].x * f, acc[v].y * f, acc[v].z * f, acc[v].w * f);
        tot *= f;
        m_run = top;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float w = exp2f(l[i] - ref);
            if (w == 0.0f) continue;                                     // its values do not count
            tot += w;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                acc[v].x = fmaf(w, o[i][v].x, acc[v].x);
                acc[v].y = fmaf(w, o[i][v].y, acc[v].y);
                acc[v].z = fmaf(w, o[i][v].z, acc[v].z);
                acc[v].w = fmaf(w, o[i][v].w, acc[v].w);
            }
        }
    }
    const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
#pragma unroll
    for (int v = 0; v < V; ++v)
        *reinterpret_cast<uint2*>(out + (m.out_row + row) * kValueDim + d0 + v * 128 + lane * 4) =
            make_uint2(pack_bf16x2(acc[v].x * inv, acc[v].y * inv), pack_bf16x2(acc[v].z * inv, acc[v].w * inv));
    if (lse_out != nullptr && d0 == 0 && lane == 0)
        lse_out[m.out_row + row] = tot == 0.0f ? -INFINITY : (m_run + log2f(tot)) * kLn2;
}

__global__ void __launch_bounds__(kCombThreads)
dense_mla_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                         const Meta* __restrict__ meta, int clusters, int slot_rows, uint16_t* __restrict__ out,
                         float* __restrict__ lse_out) {
    // the row tiles to join, read at once (one after the other they would cost a memory latency each) and
    // listed in order, so that every block counts alike
    __shared__ Meta list[kCombThreads];
    __shared__ int list_c[kCombThreads], found[kCombThreads / 32];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nwarps = gridDim.x * (kCombThreads / 32);
    const int first = blockIdx.x * (kCombThreads / 32) + warp;
    for (int c0 = 0; c0 < clusters; c0 += kCombThreads) {
        Meta own{0, 0, 0};
        if (c0 + static_cast<int>(threadIdx.x) < clusters) own = meta[c0 + threadIdx.x];
        const uint32_t mask = __ballot_sync(0xffffffffu, own.rows > 0);
        if (lane == 0) found[warp] = __popc(mask);
        __syncthreads();
        int total = 0, before = 0;
        for (int i = 0; i < kCombThreads / 32; ++i) {
            if (i == warp) before = total;
            total += found[i];
        }
        if (own.rows > 0) {
            const int j = before + __popc(mask & ((1u << lane) - 1u));
            list[j] = own;
            list_c[j] = c0 + threadIdx.x;
        }
        __syncthreads();
        const bool many = total * slot_rows >= nwarps;
        int at = first;                                                   // this warp's next task, counted over the list
        for (int li = 0; li < total; ++li) {
            const Meta m = list[li];
            const int c = list_c[li];
            const int tasks = many ? m.rows : m.rows * 4;
            for (; at < tasks; at += nwarps) {
                if (many) join_row<4, 2>(part_o, part_lse, m, c, slot_rows, at, 0, lane, out, lse_out);
                else join_row<1, 4>(part_o, part_lse, m, c, slot_rows, at >> 2, (at & 3) * 128, lane, out, lse_out);
            }
            at -= tasks;
        }
        __syncthreads();
    }
}

int decode_clusters() { return std::max(1, device_sm_count() / 2); }
int decode_slot_rows(int64_t T, int64_t H) { return static_cast<int>(std::min<int64_t>(kRows, T * H)); }

}  // namespace
}  // namespace dsa

extern "C" size_t dsa_dense_mla_decode_workspace_size(int32_t T, int32_t H) {
    using namespace dsa;
    if (T <= 0 || H <= 0) return 0;
    const size_t c = static_cast<size_t>(decode_clusters()), rows = static_cast<size_t>(decode_slot_rows(T, H));
    return c * sizeof(Meta) + 2 * c * rows * (kValueDim + 1) * sizeof(float);
}

extern "C" dsa_status dsa_dense_mla_decode(const void* q_bf16, const void* kv_pool, int64_t num_pages,
                                           const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                                           const int32_t* cu_q, int32_t B, int32_t T, int32_t H, float scale,
                                           void* out_bf16, float* lse, void* workspace, size_t workspace_bytes,
                                           int32_t* dev_err, void* stream) {
    using namespace dsa;
    if (H != 16 && H != 32 && H != 64 && H != 128) return DSA_ERR_UNSUPPORTED;
    if (T < 0 || B < 0 || max_pages < 0 || num_pages < 0) return DSA_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return DSA_OK;
    if (num_pages < 1 || max_pages < 1) return DSA_ERR_INVALID_ARG;
    if (!q_bf16 || !kv_pool || !block_table || !seq_lens || !cu_q || !out_bf16) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_bf16) || !aligned16(kv_pool) || !aligned16(out_bf16)) return DSA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !(scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    if ((num_pages + 1) * kPage >= 0x7fffffffLL || static_cast<int64_t>(max_pages) * kPage >= 0x7fffffffLL ||
        static_cast<int64_t>(T) * H >= 0x7fffffffLL || B > kMaxRequests)
        return DSA_ERR_UNSUPPORTED;
    // the schedule counts key tiles in 32 bits
    if (static_cast<int64_t>(T) * max_pages >= 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
    const size_t need = dsa_dense_mla_decode_workspace_size(T, H);
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need) return DSA_ERR_INVALID_ARG;
    auto encode = attn::tensor_map_encoder();
    if (encode == nullptr) return DSA_ERR_CUDA;
    const int clusters = decode_clusters(), slot_rows = decode_slot_rows(T, H);
    Meta* meta = static_cast<Meta*>(workspace);
    float* part_o = reinterpret_cast<float*>(meta + clusters);
    float* part_lse = part_o + static_cast<size_t>(2) * clusters * slot_rows * kValueDim;
    CUtensorMap kvmap, qmap, omap, pmap;
    if (!attn::encode_bf16_3d(encode, &kvmap, kv_pool, kLatentDim, 1, num_pages * kPage, kLatentDim, kLatentDim, 64, kPage) ||
        !attn::encode_bf16_3d(encode, &qmap, q_bf16, kLatentDim, 1, static_cast<uint64_t>(T) * H, kLatentDim, kLatentDim, 64, kRows) ||
        !attn::encode_bf16_3d(encode, &omap, out_bf16, kValueDim, 1, static_cast<uint64_t>(T) * H, kValueDim, kValueDim, 64, 16) ||
        !attn::encode_f32_rows(encode, &pmap, part_o, kValueDim, static_cast<uint64_t>(2) * clusters * slot_rows, 32, 16))
        return DSA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaFuncSetAttribute(dense_mla_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kDecSmem)) != cudaSuccess)
        return DSA_ERR_CUDA;
    // both kernels are programmatic dependents: scheduled as the CTAs of the one before end, they wait for all of it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters);
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = kDecSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dense_mla_decode_kernel, kvmap, qmap, omap, pmap, static_cast<const uint16_t*>(kv_pool),
                           static_cast<int>(num_pages), block_table, Batch{seq_lens, cu_q, B, T, H, max_pages, kRows / H},
                           scale, static_cast<uint16_t*>(out_bf16), lse, part_lse, meta, slot_rows, dev_err) != cudaSuccess)
        return DSA_ERR_CUDA;
    cfg.gridDim = dim3(2 * clusters * kCombBlocks);
    cfg.blockDim = dim3(kCombThreads);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, dense_mla_combine_kernel, static_cast<const float*>(part_o),
                           static_cast<const float*>(part_lse), static_cast<const Meta*>(meta), clusters, slot_rows,
                           static_cast<uint16_t*>(out_bf16), lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}
