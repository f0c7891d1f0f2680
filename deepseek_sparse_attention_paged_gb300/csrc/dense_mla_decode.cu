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
// the key takes, and its output accumulator (128 x 512 fp32) alone would fill the tensor memory.  So
// two CTAs of a cluster share a row tile: rank c owns the value dims 256 c .. 256 c + 255 and the rope
// dims 512 + 32 c .. 512 + 32 c + 31, reads only those of every cached row, forms the partial scores
// over them and accumulates its own 256 output dims.  The softmax is split by rows: rank c owns the
// 32-row groups c and c + 2; it receives the peer's partial scores of them (fp32, st.async into its
// shared memory), and sends P (bf16) and the rescaling factors back.  That is 24 KB a tile and
// direction over the cluster network (about 32 bytes a cycle), where a swap of all partial scores
// took 32 KB and the whole softmax in both CTAs.
//
// Work: the key tiles (64 positions = one page) of all row tiles in one sequence, cut into equal shares,
// one per cluster (at least kMinShare tiles).  A row tile that lies within one share is written
// directly; the pieces of the others go to the workspace and the combine kernel joins them.
//
// Roles (384 threads):
//   warps 0-7  rows: warp w has the rows (tensor-memory lanes) 32 (w % 4) .. + 31 and key half w / 4.
//              Owned rows: own scores + the peer's, softmax, P to both CTAs' shared memory.  Other
//              rows: partial scores to the peer, O rescaled by the peer's factors.  Queries into
//              tensor memory; output of 128 of the 256 dims at a row tile's end;
//   warp 8     TMA: the CTA's dims of each page, 4 chunks of 64 value dims and 32 rope dims, 4-deep ring;
//   warp 9     MMA: S = Q K^T (A in tensor memory, rope part in shared memory), two tiles ahead, and
//              O += P V (P in shared memory), whichever is ready; warps 10 and 11 idle.
// Tensor memory: O (columns 0-255), two score tiles (256-383), the CTA's 4 query chunks (384-511).
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"

namespace dsa {
namespace {

using namespace attn;

constexpr int kRows = 128;                                      // query rows of a row tile (MMA M)
constexpr int kKeys = 64;                                       // keys of a tile: one page
constexpr int kChunks = 4;                                      // value chunks (64 dims) per CTA
constexpr int kChunkBytes = kKeys * 128;                        // 8192, 128-byte swizzle
constexpr int kRopeBytes = kKeys * 64;                          // 4096, 64-byte swizzle
constexpr int kStageBytes = kChunks * kChunkBytes + kRopeBytes; // 36864
constexpr int kStages = 4;
constexpr int kOwnRows = kRows / 2;                             // rows whose softmax a CTA takes
constexpr int kXBytes = kOwnRows * kKeys * 4;                   // 16384: the peer's partial scores of them
constexpr int kPBytes = kRows * kKeys * 2;                      // 16384: P, K-major, 128-byte swizzle
constexpr int kQRopeBytes = kRows * 64;                         // 8192
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kDecThreads = 384;
constexpr uint32_t kColS = 256, kColQ = 384;
constexpr int kHalf = kValueDim / 2;
constexpr int kMaxRequests = 16384;                             // prefix sums of the schedule fit the ring
constexpr int kMinShare = 4;
constexpr size_t kDecSmem = 1024 + size_t(kStages) * kStageBytes + 2 * size_t(kXBytes + kPBytes) + kQRopeBytes + 4096;
static_assert(kDecSmem <= 232448, "shared-memory budget");
static_assert(kMaxRequests * 4 <= kStages * kStageBytes, "schedule scratch");

struct DecBars {
    uint64_t q_full;                        // queries in place (8 row warps), per row tile
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t s_full[2];                     // partial scores complete
    uint64_t s_read[2];                     // ... and read (8 row warps)
    uint64_t x_full[2];                     // the peer's partial scores of the owned rows arrived (armed + bytes)
    uint64_t x_free[2];                     // the peer has read the ones sent to it (its 4 owning warps)
    uint64_t pair[2];                       // both key halves of an owned row group have written (2 warps)
    uint64_t p_full[2];                     // P in place: 4 owning warps here, armed + bytes from the peer
    uint64_t a_full[2];                     // the peer's rescaling factors arrived (armed + bytes)
    uint64_t scaled[2];                     // O of the other rows rescaled by them (4 warps)
    uint64_t pv_done[2];                    // P V of the tile complete in both CTAs
    uint64_t o_free;                        // O read out (8 row warps), per row tile
    uint64_t fin_full;                      // the peer's 1 / l arrived (armed + bytes), per row tile
    uint32_t tmem_slot;
    int page_ok[kStages];                   // the stage's page id was valid
    int start[4];                           // first request, first row tile of it, first key tile, tiles of the share
    int first_cluster;                      // cluster that holds the first piece of the first row tile
    float tmax[2][2][kOwnRows];             // [tile parity][key half][owned row]: maximum of the tile
    float lsum[2][kOwnRows];                // [key half]: sums at a row tile's end
    float alpha[2][kOwnRows];               // [tile parity]: the peer's factors of the other rows
    float fin[kOwnRows];                    // the peer's 1 / l of the other rows; -1: nothing visible
};
static_assert(sizeof(DecBars) <= 4096, "barrier block");

struct Batch {
    const int32_t* seq_lens;
    const int32_t* cu_q;
    int B, T, H, max_pages;
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

__device__ __forceinline__ RowTile row_tile(const Batch& bt, int L, int q0, int nq, int g) {
    const int per = kRows / bt.H;
    RowTile t;
    t.row0 = q0 + g * per;
    t.tokens = min(per, nq - g * per);
    t.vis0 = L - nq + g * per + 1;
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
        L = uniform(__ldg(bt.seq_lens + b));
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
        if ((g + 1) * (kRows / bt.H) < nq) {
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
    const int L = __ldg(bt.seq_lens + b);
    int sum = 0;
    for (int g = 0; g * (kRows / bt.H) < nq; ++g) {
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
                        const int L = __ldg(bt.seq_lens + b);
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
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared::cluster address of the same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t smem_addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}
// 16-byte store into another CTA's shared memory, counted as transaction bytes on that CTA's
// mbarrier (the receiver's wait on it orders the data).
__device__ __forceinline__ void st_async_f32(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
// Arrive on a barrier of the peer without ordering anything before it: used for buffers this thread has
// only read (the values are in registers).  A release at cluster scope costs about 2000 cycles here.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs issued so far have completed.
__device__ __forceinline__ void umma_commit_both(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Descriptor of a K-major operand with the 64-byte swizzle: rows of 64 bytes, 8-row groups 512 apart.
__device__ __forceinline__ uint64_t desc_sw64(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>(512u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(4u) << 61;
    return d;
}

// What a cluster leaves for the combine kernel: the split row tile whose last piece it computed.
struct Meta {
    int64_t out_row;       // first output row (token * H)
    int rows;              // its rows; 0: none
    int first_cluster;
};

__global__ void __launch_bounds__(kDecThreads, 1) __cluster_dims__(2, 1, 1)
dense_mla_decode_kernel(const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap rmap,
                        const uint16_t* __restrict__ q, int num_pages, const int32_t* __restrict__ block_table,
                        Batch bt, float scale, uint16_t* __restrict__ out, float* __restrict__ lse_out,
                        float* __restrict__ part_o, float* __restrict__ part_lse, Meta* __restrict__ meta, int slot_rows,
                        int32_t* err) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    unsigned char* ring = base;
    unsigned char* ps = ring + kStages * kStageBytes;                              // [2][128 rows][64 keys], 128-byte swizzle
    float* xs = reinterpret_cast<float*>(ps + 2 * kPBytes);                        // [2][16 key quads][64 rows][4]
    unsigned char* qrope = reinterpret_cast<unsigned char*>(xs) + 2 * kXBytes;     // [128 rows][32 dims], 64-byte swizzle
    DecBars& bar = *reinterpret_cast<DecBars*>(qrope + kQRopeBytes);

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank(), peer = crank ^ 1u;
    const int half = static_cast<int>(crank);
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        ptx::mbar_init(&bar.q_full, 8);
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bar.kv_full[s], 1);
            ptx::mbar_init(&bar.kv_empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&bar.s_full[a], 1);
            ptx::mbar_init(&bar.s_read[a], 8);
            ptx::mbar_init(&bar.x_full[a], 1);
            ptx::mbar_init(&bar.x_free[a], 4);
            ptx::mbar_init(&bar.pair[a], 2);
            ptx::mbar_init(&bar.p_full[a], 5);
            ptx::mbar_init(&bar.a_full[a], 1);
            ptx::mbar_init(&bar.scaled[a], 4);
            ptx::mbar_init(&bar.pv_done[a], 2);
        }
        ptx::mbar_init(&bar.o_free, 8);
        ptx::mbar_init(&bar.fin_full, 1);
        ptx::fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&bar.tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    find_share(bt, cluster, clusters, reinterpret_cast<int*>(ring), bar, half == 0 ? err : nullptr);
    ptx::fence_proxy_async_smem();   // the schedule's scratch lies where copies will land
    ptx::tc_fence_before_sync();
    cluster_sync_all();              // both CTAs' barriers exist before the peer signals or writes into them
    ptx::tc_fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem_slot);
    const uint64_t deadline = ptx::wait_deadline();
    bool timed_out = false;
    const bool work = uniform(bar.start[3]) > 0;

    if (warp == kTmaWarp) {
        // ---------------------------------------------------------------- TMA
        if (work) {
            Walk w(bt, bar.start);
            uint32_t it = 0;
            do {
                int page = -1;
                for (int t = w.t0; t < w.t1 && !timed_out; ++t, ++it) {
                    if (((t - w.t0) & 31) == 0)                      // page ids of the next 32 tiles
                        page = t + lane < w.t1 ? __ldg(block_table + static_cast<int64_t>(w.b) * bt.max_pages + t + lane) : 0;
                    const int pg = __shfl_sync(0xffffffffu, page, (t - w.t0) & 31);
                    const int s = static_cast<int>(it % kStages);
                    if (lane == 0) {
                        const bool ok = pg >= 0 && pg < num_pages;
                        // a page outside the pool: a box past the end reads zeros, and nothing of it counts
                        const int row = (ok ? pg : num_pages) * kPage;
                        if (!ok) raise_error(err, DSA_DEVERR_PAGE_RANGE);
                        if (!ptx::mbar_wait(&bar.kv_empty[s], ((it / kStages) & 1u) ^ 1u, deadline)) {
                            timed_out = true;
                        } else {
                            bar.page_ok[s] = ok ? 1 : 0;
                            ptx::mbar_arrive_expect_tx(&bar.kv_full[s], kStageBytes);
                            unsigned char* st = ring + s * kStageBytes;
#pragma unroll
                            for (int j = 0; j < kChunks; ++j)
                                ptx::tma_load_3d(st + j * kChunkBytes, &vmap, &bar.kv_full[s], half * kHalf + 64 * j, 0, row);
                            ptx::tma_load_3d(st + kChunks * kChunkBytes, &rmap, &bar.kv_full[s], kValueDim + half * 32, 0, row);
                        }
                    }
                    timed_out = __any_sync(0xffffffffu, timed_out);
                }
            } while (!timed_out && w.next());
            // copies still in flight land before the CTA may leave (bounded)
            if (lane == 0)
                for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
                    if (!ptx::mbar_wait(&bar.kv_full[j % kStages], (j / kStages) & 1u, ptx::wait_deadline(20000000ull)))
                        timed_out = true;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA
        if (work) {
            constexpr uint32_t idesc_qk = ptx::instr_desc(1, 1, kRows, kKeys);
            constexpr uint32_t idesc_pv = ptx::instr_desc(1, 1, kRows, kHalf) | (1u << 16);   // B MN-major
            const uint32_t ring_addr = ptx::smem_addr(ring);
            const uint64_t k_desc = desc_sw128(ring_addr, 16, 1024), v_desc = desc_sw128(ring_addr, kChunkBytes, 1024);
            const uint64_t r_desc = desc_sw64(ring_addr + kChunks * kChunkBytes), qr_desc = desc_sw64(ptx::smem_addr(qrope));
            // a wait that ran out only marks the step; the warp leaves at the step's end
            bool late = false;
            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (!ptx::mbar_wait(b, parity, deadline)) late = true;
            };
            const uint64_t p_desc = desc_sw128(ptx::smem_addr(ps), 16, 1024);
            Walk w(bt, bar.start);
            uint32_t it = 0, seg = 0;                                // tiles of the pieces before; pieces with tiles
            do {
                if (w.t0 >= w.t1) continue;
                const int live = w.rt.tokens * bt.H;
                const uint32_t peer_quads = (static_cast<int>(peer) * 32 < live ? 1u : 0u) +
                                            (static_cast<int>(peer + 2) * 32 < live ? 1u : 0u);
                const uint32_t n = static_cast<uint32_t>(w.t1 - w.t0);
                uint32_t iq = 0, ip = 0;                             // next score tile, next P V tile of the piece
                wait(&bar.q_full, seg & 1u);
                while (ip < n) {
                    bool issued = false;
                    // scores of tile iq: keys landed, the score buffer read
                    if (iq < n && iq < ip + 2) {
                        const uint32_t u = it + iq, s = u % kStages;
                        const bool ready = ptx::mbar_test_wait(&bar.kv_full[s], (u / kStages) & 1u) &&
                                           (u < 2 || ptx::mbar_test_wait(&bar.s_read[u & 1], ((u >> 1) & 1u) ^ 1u));
                        if (__all_sync(0xffffffffu, ready)) {
                            const int valid = w.rt.vis0 + w.rt.tokens - 1 - (w.t0 + static_cast<int>(iq)) * kKeys;
                            if (valid < kKeys) {
                                // rows past the last visible position may hold anything: their P is 0, but
                                // 0 times NaN or infinity is not
                                unsigned char* st = ring + s * kStageBytes;
                                for (int e = lane; e < (kKeys - valid) * 8; e += 32)
#pragma unroll
                                    for (int j = 0; j < kChunks; ++j)
                                        *reinterpret_cast<uint4*>(st + j * kChunkBytes + (valid + (e >> 3)) * 128 + (e & 7) * 16) =
                                            make_uint4(0u, 0u, 0u, 0u);
                                ptx::fence_proxy_async_smem();
                                __syncwarp();
                            }
                            ptx::tc_fence_after_sync();
                            if (elect_one()) {
                                // the previous phase is over: the P V of tile u - 2 has been issued
                                ptx::mbar_arrive_expect_tx(&bar.p_full[u & 1], peer_quads * (32 * kKeys * 2));
                                const uint64_t so = s * (kStageBytes / 16);
                                const uint32_t d = tmem + kColS + (u & 1) * kKeys;
#pragma unroll
                                for (int j = 0; j < kChunks; ++j)
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        umma_f16_ts(d, tmem + kColQ + j * 32 + kk * 8, k_desc + so + j * (kChunkBytes / 16) + kk * 2,
                                                    idesc_qk, (j | kk) != 0 ? 1u : 0u);
#pragma unroll
                                for (int kk = 0; kk < 2; ++kk)
                                    ptx::umma_f16(d, qr_desc + kk * 2, r_desc + so + kk * 2, idesc_qk, 1u);
                                ptx::umma_commit(&bar.s_full[u & 1]);
                            }
                            __syncwarp();
                            ++iq;
                            issued = true;
                        }
                    }
                    // O += P V of tile ip: P in place, the other rows rescaled, O of the previous row tile read out
                    if (ip < iq) {
                        const uint32_t u = it + ip, ph = (u >> 1) & 1u;
                        const bool ready = ptx::mbar_test_wait(&bar.p_full[u & 1], ph) && ptx::mbar_test_wait(&bar.scaled[u & 1], ph) &&
                                           (ip > 0 || seg == 0 || ptx::mbar_test_wait(&bar.o_free, (seg - 1) & 1u));
                        if (__all_sync(0xffffffffu, ready)) {
                            ptx::fence_proxy_async_smem();           // P comes from ordinary and st.async stores
                            ptx::tc_fence_after_sync();
                            if (elect_one()) {
                                const uint64_t vb = v_desc + (u % kStages) * (kStageBytes / 16);
                                const uint64_t pb = p_desc + (u & 1) * (kPBytes / 16);
#pragma unroll
                                for (int ks = 0; ks < kKeys / 16; ++ks)
                                    ptx::umma_f16(tmem, pb + ks * 2, vb + ks * 128, idesc_pv, (ip | ks) != 0 ? 1u : 0u);
                                ptx::umma_commit(&bar.kv_empty[u % kStages]);
                                umma_commit_both(&bar.pv_done[u & 1]);
                            }
                            __syncwarp();
                            ++ip;
                            issued = true;
                        }
                    }
                    if (!issued && static_cast<uint64_t>(clock64()) > deadline) late = true;
                    if (__any_sync(0xffffffffu, late)) break;
                }
                it += n;
                ++seg;
            } while (!__any_sync(0xffffffffu, late) && w.next());
            if (late) timed_out = true;
        }
    } else if (warp < kTmaWarp) {
        // ---------------------------------------------------------------- rows
        if (threadIdx.x == 0 && half == 0) meta[cluster].rows = 0;
        if (work) {
            const int quad = warp & 3, kh = warp >> 2;
            const int row = quad * 32 + lane;                        // query row of the row tile = tensor-memory lane
            const bool own = (quad & 1) == half;
            const int place = (quad >> 1) * 32 + lane;               // among the owned / the other rows
            const bool lead = (quad >> 1) == 0 && kh == 0 && lane == 0;   // arms this side's barriers
            const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
            const uint32_t o_addr = tmem + lane_base + kh * 128;     // this warp's 128 of the CTA's 256 output dims
            const float cs = scale * kLog2e;
            const uint64_t cs2 = f32x2(cs, cs);
            const int token = row / bt.H;
            const uint32_t peer_p = map_to_rank(ptx::smem_addr(ps), peer);
            const uint32_t peer_x = map_to_rank(ptx::smem_addr(xs), peer) + place * 16 + kh * 8 * (kOwnRows * 16);
            uint32_t p_off[4];                                       // the row's 16-byte pieces of this key half
#pragma unroll
            for (int i = 0; i < 4; ++i) p_off[i] = row * 128 + (((kh * 4 + i) ^ (row & 7)) << 4);
            uint32_t it = 0, seg = 0, meets = 0;                     // meets: uses of the pair barrier
            bool q_loaded = false;

            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (!ptx::mbar_wait(b, parity, deadline)) timed_out = true;
            };
            // a row tile's queries: value chunks 2 kh, 2 kh + 1 into tensor memory, rope pieces 2 kh, 2 kh + 1
            // into shared memory (the score MMAs before are complete: their s_full has been waited for)
            auto load_q = [&](const RowTile& rt) {
                const int n = rt.tokens * bt.H;
                if (quad * 32 < n) {
                    const uint4* src = reinterpret_cast<const uint4*>(
                        q + (static_cast<int64_t>(rt.row0) * bt.H + row) * kLatentDim);
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 r = row < n ? __ldg(src + half * (kHalf / 8) + (2 * kh + j) * 8 + i) : zero;
                            v[4 * i] = r.x; v[4 * i + 1] = r.y; v[4 * i + 2] = r.z; v[4 * i + 3] = r.w;
                        }
                        tmem_st_x32(tmem + lane_base + kColQ + (2 * kh + j) * 32, v);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<uint4*>(qrope + row * 64 + (((2 * kh + j) ^ ((row >> 1) & 3)) << 4)) =
                            row < n ? __ldg(src + (kValueDim + half * 32) / 8 + 2 * kh + j) : zero;
                    ptx::fence_proxy_async_smem();
                    tmem_wait_st();
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.q_full);
            };
            // this warp's part of O times alpha, before tile u is added, once the tiles before are
            auto rescale = [&](float alpha, uint32_t u) {
                wait(&bar.pv_done[(u - 1) & 1u], ((u - 1) >> 1) & 1u);
                __syncwarp();
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int cc = 0; cc < 128; cc += 32) {
                    uint32_t o[32];
                    ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st_x32(o_addr + cc, o);
                }
                tmem_wait_st();
            };
            // other rows: tile u's partial scores to the peer
            auto send = [&](uint32_t u, bool live) {
                const uint32_t bb = u & 1u, ph = (u >> 1) & 1u;
                wait(&bar.s_full[bb], ph);
                if (live) {
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(tmem + lane_base + kColS + bb * kKeys + kh * 32, v);
                    if (u >= 2) wait(&bar.x_free[bb], ph ^ 1u);
                    ptx::tmem_wait_ld();
                    const uint32_t dst = peer_x + bb * kXBytes, xb = map_to_rank(ptx::smem_addr(&bar.x_full[bb]), peer);
#pragma unroll
                    for (int k4 = 0; k4 < 8; ++k4)
                        st_async_v4(dst + k4 * (kOwnRows * 16), v[4 * k4], v[4 * k4 + 1], v[4 * k4 + 2], v[4 * k4 + 3], xb);
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.s_read[bb]);
            };

            Walk w(bt, bar.start);
            for (;;) {
                const int live = w.rt.tokens * bt.H;
                const bool quad_live = quad * 32 < live;
                const uint32_t my_quads = (half * 32 < live ? 1u : 0u) + ((half + 2) * 32 < live ? 1u : 0u);
                const uint32_t peer_quads = (static_cast<int>(peer) * 32 < live ? 1u : 0u) +
                                            (static_cast<int>(peer + 2) * 32 < live ? 1u : 0u);
                const int vis = min(w.rt.vis0 + token, bt.max_pages * kPage);
                const bool has_tiles = w.t0 < w.t1;
                float m_run = -INFINITY, l_run = 0.0f;
                if (has_tiles && !q_loaded) load_q(w.rt);
                if (!own) {
                    const int n = w.t1 - w.t0;
                    if (n > 0) send(it, quad_live);
                    for (int i = 0; i < n; ++i, ++it) {
                        const uint32_t bb = it & 1u, ph = (it >> 1) & 1u;
                        if (i + 1 < n) send(it + 1, quad_live);
                        if (lead) ptx::mbar_arrive_expect_tx(&bar.a_full[bb], peer_quads * 128);
                        wait(&bar.a_full[bb], ph);
                        if (quad_live && i > 0) {
                            const float alpha = bar.alpha[bb][place];
                            if (__any_sync(0xffffffffu, alpha != 1.0f)) rescale(alpha, it);
                        }
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&bar.scaled[bb]);
                        timed_out = __any_sync(0xffffffffu, timed_out);
                        if (timed_out) break;
                    }
                } else {
                    for (int t = w.t0; t < w.t1; ++t, ++it) {
                        const uint32_t bb = it & 1u, ph = (it >> 1) & 1u;
                        const int s = static_cast<int>(it % kStages);
                        if (lead) ptx::mbar_arrive_expect_tx(&bar.x_full[bb], my_quads * (32 * kKeys * 4));
                        wait(&bar.s_full[bb], ph);
                        if (quad_live) {
                            __syncwarp();
                            ptx::tc_fence_after_sync();
                            uint32_t v[32];
                            ptx::tmem_ld_32x32b_x32(tmem + lane_base + kColS + bb * kKeys + kh * 32, v);
                            wait(&bar.kv_full[s], (it / kStages) & 1u);            // orders page_ok
                            wait(&bar.x_full[bb], ph);
                            const float* xr = xs + bb * (kXBytes / 4) + (kh * 8 * kOwnRows + place) * 4;
                            float4 x[8];
#pragma unroll
                            for (int k4 = 0; k4 < 8; ++k4) x[k4] = *reinterpret_cast<const float4*>(xr + k4 * (kOwnRows * 4));
                            ptx::tmem_wait_ld();
                            ptx::tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&bar.s_read[bb]);
                            float sc[32];
#pragma unroll
                            for (int k4 = 0; k4 < 8; ++k4) {
                                sc[4 * k4] = __uint_as_float(v[4 * k4]) + x[k4].x;
                                sc[4 * k4 + 1] = __uint_as_float(v[4 * k4 + 1]) + x[k4].y;
                                sc[4 * k4 + 2] = __uint_as_float(v[4 * k4 + 2]) + x[k4].z;
                                sc[4 * k4 + 3] = __uint_as_float(v[4 * k4 + 3]) + x[k4].w;
                            }
                            const int lim = (bar.page_ok[s] ? vis - t * kKeys : 0) - kh * 32;
                            if (lim < 32) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (e >= lim) sc[e] = -INFINITY;
                            }
                            float mx4[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
                            for (int e = 4; e < 32; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], sc[e]);
                            float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                            // the tile's maximum over both key halves (values double-buffered by tile parity)
                            bar.tmax[bb][kh][place] = mx;
                            // every lane's scores have been read (the maximum needs them): the peer may send again
                            __syncwarp();
                            if (lane == 0) {
                                ptx::mbar_arrive(&bar.pair[quad >> 1]);
                                arrive_remote(map_to_rank(ptx::smem_addr(&bar.x_free[bb]), peer));
                            }
                            wait(&bar.pair[quad >> 1], meets & 1u);
                            ++meets;
                            mx = fmaxf(mx, bar.tmax[bb][kh ^ 1][place]);
                            const bool grow = (mx - m_run) * cs > kRescaleThreshold || (m_run == -INFINITY && mx > -INFINITY);
                            float alpha = 1.0f;
                            if (__any_sync(0xffffffffu, grow)) {
                                if (grow) {
                                    alpha = m_run == -INFINITY ? 0.0f : exp2f((m_run - mx) * cs);
                                    m_run = mx;
                                }
                                l_run *= alpha;
                                if (t > w.t0) rescale(alpha, it);
                            }
                            const float neg = m_run == -INFINITY ? 0.0f : -m_run * cs;
                            const uint64_t neg2 = f32x2(neg, neg);
                            uint64_t sum2 = f32x2(0.0f, 0.0f);
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float a, b;
                                unpack_f32x2(fma_f32x2(f32x2(sc[e], sc[e + 1]), cs2, neg2), a, b);
                                a = fast_exp2(a);
                                b = fast_exp2(b);
                                sum2 = add_f32x2(sum2, f32x2(a, b));
                                pk[e / 2] = pack_bf16x2(a, b);
                            }
                            // the P V that read the buffer's previous P is complete in both CTAs
                            if (it >= 2) wait(&bar.pv_done[bb], ph ^ 1u);
                            const uint32_t pb = map_to_rank(ptx::smem_addr(&bar.p_full[bb]), peer);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                st_async_v4(peer_p + bb * kPBytes + p_off[i], pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3], pb);
                                *reinterpret_cast<uint4*>(ps + bb * kPBytes + p_off[i]) =
                                    make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                            }
                            if (kh == 0)
                                st_async_f32(map_to_rank(ptx::smem_addr(&bar.alpha[bb][place]), peer), alpha,
                                             map_to_rank(ptx::smem_addr(&bar.a_full[bb]), peer));
                            ptx::fence_proxy_async_smem();
                            float a, b;
                            unpack_f32x2(sum2, a, b);
                            l_run += a + b;
                        } else if (lane == 0) {
                            ptx::mbar_arrive(&bar.s_read[bb]);
                            arrive_remote(map_to_rank(ptx::smem_addr(&bar.x_free[bb]), peer));
                        }
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&bar.p_full[bb]);
                        timed_out = __any_sync(0xffffffffu, timed_out);
                        if (timed_out) break;
                    }
                }
                if (timed_out) break;
                // ---- the next row tile's queries, so that its first scores run during this one's output
                Walk nxt = w;
                const bool more = nxt.next();
                q_loaded = more && nxt.t0 < nxt.t1;
                if (q_loaded) load_q(nxt.rt);
                // ---- the piece's output: O / l and its log-sum-exp (log2 units for a part)
                float inv = -1.0f;                                   // -1: nothing visible (O may hold 0 x NaN)
                if (own && quad_live) {
                    float l_tot = 0.0f;
                    if (has_tiles) {
                        bar.lsum[kh][place] = l_run;
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&bar.pair[quad >> 1]);
                        wait(&bar.pair[quad >> 1], meets & 1u);
                        ++meets;
                        l_tot = l_run + bar.lsum[kh ^ 1][place];
                        if (l_tot != 0.0f) inv = 1.0f / l_tot;
                    }
                    if (kh == 0) {
                        if (has_tiles)
                            st_async_f32(map_to_rank(ptx::smem_addr(&bar.fin[place]), peer), inv,
                                         map_to_rank(ptx::smem_addr(&bar.fin_full), peer));
                        if (row < live) {
                            const float lse2 = l_tot == 0.0f ? -INFINITY : m_run * cs + log2f(l_tot);
                            if (!w.whole) part_lse[piece_slot(cluster, w) * slot_rows + row] = lse2;
                            else if (lse_out != nullptr) lse_out[static_cast<int64_t>(w.rt.row0) * bt.H + row] = lse2 * kLn2;
                        }
                    }
                } else if (!own && has_tiles) {
                    if (lead) ptx::mbar_arrive_expect_tx(&bar.fin_full, peer_quads * 128);
                    wait(&bar.fin_full, seg & 1u);
                    inv = bar.fin[place];
                }
                if (has_tiles) {
                    wait(&bar.pv_done[(it - 1) & 1u], ((it - 1) >> 1) & 1u);
                    timed_out = __any_sync(0xffffffffu, timed_out);
                    if (timed_out) break;
                    ptx::tc_fence_after_sync();
                }
                if (quad_live) {
                    const int dim = half * kHalf + kh * 128;
                    uint16_t* dst = out + (static_cast<int64_t>(w.rt.row0) * bt.H + row) * kValueDim + dim;
                    float* pdst = part_o + (piece_slot(cluster, w) * slot_rows + row) * kValueDim + dim;
#pragma unroll 1
                    for (int cc = 0; cc < 128; cc += 32) {
                        uint32_t o[32];
                        if (has_tiles) {
                            ptx::tmem_ld_32x32b_x32(o_addr + cc, o);
                            ptx::tmem_wait_ld();
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = inv < 0.0f ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
                        if (row < live) {
                            if (w.whole) {
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
                                    *reinterpret_cast<uint4*>(dst + cc + e) = make_uint4(
                                        pack_bf16x2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                                        pack_bf16x2(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                                        pack_bf16x2(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])),
                                        pack_bf16x2(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<uint4*>(pdst + cc + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                            }
                        }
                    }
                }
                if (has_tiles) {
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar.o_free);
                    ++seg;
                }
                // the last piece of a split row tile: the combine kernel finds it here
                if (threadIdx.x == 0 && half == 0 && w.first && w.t0 > 0 && w.t1 == w.rt.tiles)
                    meta[cluster] = Meta{static_cast<int64_t>(w.rt.row0) * bt.H, live, bar.first_cluster};
                if (!more) break;
                w = nxt;
            }
        }
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

// Joins the pieces of the split row tiles: one warp per (output row, 128 of its 512 dims).  The first
// piece lies in slot 2 c0 + 1, the following ones in slots 2 (c0 + 1), .., 2 c.
constexpr int kCombThreads = 256;
__global__ void __launch_bounds__(kCombThreads)
dense_mla_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                         const Meta* __restrict__ meta, int clusters, int slot_rows, uint16_t* __restrict__ out,
                         float* __restrict__ lse_out) {
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int nwarps = gridDim.x * (kCombThreads / 32);
    int at = blockIdx.x * (kCombThreads / 32) + (threadIdx.x >> 5);   // this warp's next task, counted over all row tiles
    for (int c = 0; c < clusters; ++c) {
        const Meta m = meta[c];
        const int tasks = m.rows * 4;
        for (; at < tasks; at += nwarps) {
            const int row = at >> 2, d0 = (at & 3) * 128 + lane * 4;
            const int n = c - m.first_cluster + 1;
            auto slot_of = [&](int j) {
                return static_cast<int64_t>(j == 0 ? 2 * m.first_cluster + 1 : 2 * (m.first_cluster + j)) * slot_rows + row;
            };
            float top = -INFINITY;
            bool nan = false;
            for (int j = lane; j < n; j += 32) {
                const float l = part_lse[slot_of(j)];
                top = fmaxf(top, l);
                nan |= l != l;
            }
            top = warp_max(top);
            float tot = 0.0f;
            if (top != -INFINITY)
                for (int j = lane; j < n; j += 32) tot += exp2f(part_lse[slot_of(j)] - top);
            tot = warp_sum(tot);
            if (__any_sync(0xffffffffu, nan)) tot = NAN;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (top != -INFINITY) {
                const float inv = 1.0f / tot;
#pragma unroll 4
                for (int j = 0; j < n; ++j) {
                    const int64_t s = slot_of(j);
                    const float w = exp2f(part_lse[s] - top) * inv;
                    const float4 o = *reinterpret_cast<const float4*>(part_o + s * kValueDim + d0);
                    acc.x = fmaf(w, o.x, acc.x);
                    acc.y = fmaf(w, o.y, acc.y);
                    acc.z = fmaf(w, o.z, acc.z);
                    acc.w = fmaf(w, o.w, acc.w);
                }
            }
            *reinterpret_cast<uint2*>(out + (m.out_row + row) * kValueDim + d0) =
                make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            if (lse_out != nullptr && (at & 3) == 0 && lane == 0)
                lse_out[m.out_row + row] = top == -INFINITY ? -INFINITY : (top + log2f(tot)) * kLn2;
        }
        at -= tasks;
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
    CUtensorMap vmap, rmap;
    if (!attn::encode_bf16_3d(encode, &vmap, kv_pool, kLatentDim, 1, num_pages * kPage, kLatentDim, kLatentDim, 64, kKeys) ||
        !attn::encode_bf16_3d(encode, &rmap, kv_pool, kLatentDim, 1, num_pages * kPage, kLatentDim, kLatentDim, 32, kKeys,
                              CU_TENSOR_MAP_SWIZZLE_64B))
        return DSA_ERR_CUDA;
    const int clusters = decode_clusters(), slot_rows = decode_slot_rows(T, H);
    Meta* meta = static_cast<Meta*>(workspace);
    float* part_o = reinterpret_cast<float*>(meta + clusters);
    float* part_lse = part_o + static_cast<size_t>(2) * clusters * slot_rows * kValueDim;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaFuncSetAttribute(dense_mla_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kDecSmem)) != cudaSuccess)
        return DSA_ERR_CUDA;
    dense_mla_decode_kernel<<<2 * clusters, kDecThreads, kDecSmem, s>>>(
        vmap, rmap, static_cast<const uint16_t*>(q_bf16), static_cast<int>(num_pages), block_table,
        Batch{seq_lens, cu_q, B, T, H, max_pages}, scale, static_cast<uint16_t*>(out_bf16), lse, part_o, part_lse, meta,
        slot_rows, dev_err);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
    // a programmatic dependent of the attention kernel: scheduled as its CTAs end, waits for all of it
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters);
    cfg.blockDim = dim3(kCombThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dense_mla_combine_kernel, static_cast<const float*>(part_o),
                           static_cast<const float*>(part_lse), static_cast<const Meta*>(meta), clusters, slot_rows,
                           static_cast<uint16_t*>(out_bf16), lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}
