// dense_mla_shared.cu -- absorbed latent attention of new tokens over the paged latent cache for batches in which groups
// of requests have their first pages in common (sm_103a).
//
// Mathematics of dense_mla_decode.cu: per row o = sum_k 2^(s_k - m) v_k / sum_k 2^(s_k - m), in one pass with a running m.
//
// Work: the query tokens of a group in units of 256 rows (heads x tokens, tokens of several requests one after the
// other).  A unit's keys are the pages of the prefix, which all of its rows see, then the pages that each of its
// requests has behind it, one request's after the other's, each row masked to its own request's.  So the
// prefix is read once for 256 rows, and requests with few heads fill the rows behind it too; nothing has to be joined
// but the pieces of a unit that is split.  The products with a page behind the prefix go into the rows of that page's request
// alone: the weights of the other rows are 0 there, but 0 times an infinite or NaN value is NaN.  (Compared with products into
// all rows: 4 requests 24.9 -> 25.2 us, 32 of 128 heads 120.3 -> 121.0, 200 behind 131008 keys 662 -> 665, others the same.)
// Requests outside all groups make up groups without a prefix.  The key tiles (128 positions = two pages) of all units in one
// sequence are cut into equal shares, one per cluster.
//
// Bound: the tensor cores, 2176 FLOP a row and key, once a prefix has about 6 rows of 16 heads.  A unit is a pipeline
// over the four CTAs of a cluster: the pair of ranks 0 and 1 forms the scores of 2 x 128 rows and their softmax, the pair
// of ranks 2 and 3 accumulates the 512 output dims (128 x 512 fp32 fill the tensor memory of an SM).  The products
// run over both SMs of a pair (M = 256), and each SM holds half of the keys' operand: one page of two for the
// scores, half of the dims for the output.  That is what the split is for: with 128 rows to a pair and its keys
// whole in each SM (the plain call) the copies in flight (128 KB an SM) cover 2300 cycles of products, less than
// they take, and a tile took 3300 cycles whether both pairs read the same tile (multicast) or not; halves cover twice that.
//
// A tile of a long prefix takes about 2800 cycles, 82 % of the nominal rate of its products, which is what the library's bf16
// product reaches on this GPU (81 %); more stages, more buffers for P or two groups of softmax warps in turn change nothing.
// Behind the prefix a tile costs the same for the few rows that see it.
//
// Measured (calls in a captured graph; in brackets the plain call on the same batch):
//   200 requests of 16 heads behind 131008 common keys     650 to 665 us (3780 to 4160), 1.38 to 1.41 PFLOP/s of what is
//                                                                 needed, 72 to 74 % of the measured rate; power
//   64 of 16 heads behind 32768, with 64 to 4096 of their own     106 us (328)
//   60 of 32 heads, two rows each, behind 5 of 2K to 32K           97 us (99)
//   32 of 128 heads behind 16384                                  120 us (119)    a request fills a tile by itself
//   4 of 16 heads behind 1024                                      25 us (20)     a chain of about 20 steps
// So it is for many requests of few heads behind one long prefix; prefixes that the L2 holds cost the plain call little where
// its own row tiles are full.  144 of 152 SMs: clusters of four do not fill a GPC whose SMs are no multiple of four.
//
// Roles (384 threads; warp 10 of each rank finds the units for the others, warp 11 is idle); "leader": the pair's even
// rank, whose MMA warp issues for both:
//   score pair  warps 0-7  softmax: rows (tensor-memory lanes) 32 (w % 4) .. + 31, page w / 4 of the tile; queries
//                          into tensor memory (value dims) and shared memory (rope dims);
//               warp 8     TMA: the rank's page, 9 chunks of 64 dims a tile;
//               warp 9     leader: S = Q K^T (N = 128) into two score tiles in turn; else gives stages back.
//   value pair  warps 0-7  O rescaled where a factor is not 1; O / l to the output, 256 dims a warp;
//               warp 8     TMA: of each 256 value dims of a page the rank's 128;
//               warp 9     leader: O += P V, one N = 256 half per stage; else tells the leader what has arrived here.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "mla_join.cuh"

namespace dsa {
namespace {

using namespace attn;

constexpr int kRows = 128;                                      // query rows of a CTA; 256 of a pair (MMA M)
constexpr int kKeys = 128;                                      // keys of a tile: two pages
constexpr int kPageChunk = kPage * 128;                         // 8192: 64 keys x 64 dims, 128-byte swizzle
constexpr int kKStageBytes = kPageChunk, kKStages = 16;         // scores: 64 dims of the rank's page; a tile is 9 stages
constexpr int kVStageBytes = 2 * kPageChunk, kVStages = 8;      // values: 128 of 256 dims of a page; a tile is 4 stages
constexpr int kMaxStages = 16;
constexpr int kLent = 4;                                        // value stages for the output: two buffers of 8 x 4 KB
constexpr int kQStages = 18;                                    // the queries, 64 rows x 64 dims a stage
constexpr int kSBufs = 2, kPBufs = 4;                           // score tiles; P buffers of one page
constexpr int kPvBars = 4, kInfo = 8;
constexpr int kPBytes = kRows * kPage * 2;                      // 16384: P of a page, K-major, 128-byte swizzle
constexpr int kQRopeBytes = kRows * 128;                        // 16384
constexpr int kPOffset = kKStages * kKStageBytes + kQRopeBytes; // P at the same place in all ranks
constexpr int kDataBytes = kPOffset + kPBufs * kPBytes;
static_assert(kVStages * kVStageBytes <= kPOffset, "value stages");
constexpr int kTmaWarp = 8, kMmaWarp = 9, kWalkWarp = 10;
constexpr int kReaders = 10;                                    // warps that walk the pieces: 0 - 9
constexpr int kPieces = 3, kUnitTokens = 16;                    // pieces known ahead; tokens of a unit
constexpr int kThreads = 384;
constexpr uint32_t kColS = 256;                                 // scores: score tiles, behind the query chunks
constexpr int kMinShare = 2;
constexpr int kUnitCost = 8;                                    // tiles that the change to another unit takes as long as (64 requests 0: 119 us,
                                                                // 4: 107; 32 requests of 128 heads 4: 124, 8: 121, 12: 123),
constexpr int kLongShare = 8;                                   // counted in shares of this many tiles or more
constexpr int kAhead = 2;                                       // tiles between a page's prefetch and its copy
constexpr int kMaxRequests = 16384, kMaxGroups = 8192, kMaxUnits = 16384;   // units of 256 rows
constexpr size_t kBarBytes = 7168;
constexpr size_t kSmem = 1024 + size_t(kDataBytes) + kBarBytes;
static_assert(kSmem <= 232448, "shared-memory budget");
static_assert((kMaxUnits + kMaxGroups + 3) * 4 <= kDataBytes, "schedule scratch");

// Where a cluster's share begins.
struct Share {
    int unit, at, left;     // first unit, where in it, length of the share
    int first;              // the cluster that holds the first piece of the first unit
    int cost;               // length of a unit in front of its tiles
};

// A piece of a share: the key tiles [t0, t1) of a unit (t0 == t1: a unit that sees nothing), and per token of the unit the
// request through whose row of the table the pages behind `prefix` are read (its own, but the prefix's first request where
// the prefix goes on), the first of its own request's pages among the unit's, how many (at the request's last token, else 0),
// and the keys it sees of the prefix and behind it.
struct Piece {
    int q0, nq, prefix, b0, pages, t0, t1;
    int whole, first;      // the piece is its whole unit; the share's first piece
    int end;               // no piece: the share is done
    int b[kUnitTokens], at[kUnitTokens], n[kUnitTokens], seen[kUnitTokens], own[kUnitTokens];
};

struct Bars {
    // leader: both CTAs' halves of the stage are there (armed + bytes); all: the stage has been read
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    // other rank: the leader is done with the stages of a unit that hold no keys (queries, output).  Until then copies into
    // such a stage here would count on the leader's barrier while that is still in the stage's earlier phase
    uint64_t lead_pass;
    // score pair
    uint64_t q_land[kQStages];              // queries in the stage (armed + bytes), per unit
    uint64_t q_read[kQStages];              // ... copied out of it (2 warps)
    uint64_t q_full;                        // leader: queries in place (16 softmax warps), per unit
    uint64_t s_full[kSBufs];                // scores complete
    uint64_t s_read[kSBufs];                // leader: ... and read (16 warps)
    uint64_t info[kInfo];                   // tile_ok written
    uint64_t pair[4];                       // both key halves of a row group have written (2 warps)
    uint64_t p_free[kPBufs];                // the P V that read the buffer is complete
    uint64_t fin_free;                      // the value rank has read 1 / l (its 8 row warps), per unit
    // value pair
    uint64_t p_full[kPBufs];                // P and the factors arrived (armed + bytes)
    uint64_t p_peer[kPBufs];                // leader: ... and in the other rank, where O is rescaled by them
    uint64_t scaled[2];                     // O rescaled by them (8 row warps), per tile
    uint64_t pv_done[kPvBars];              // P V of the tile complete (more than the tiles the row warps may be ahead)
    uint64_t o_free;                        // leader: O read out (16 row warps), per unit
    uint64_t fin_full;                      // 1 / l arrived (armed + bytes), per unit
    uint64_t stage_lent;                    // kLent ring stages are free for the output, per unit
    uint64_t stage_back;                    // ... and no longer read (8 row warps)
    uint64_t piece_full[kPieces], piece_free[kPieces];
    int stop;                               // a wait ran out somewhere in the CTA
    uint32_t tmem_slot;
    Piece piece[kPieces];
    int tile_ok[kInfo];                     // bit i: page i of the tile is there and its id valid
    Share share;
    float tmax[2][2][kRows];                // [tile parity][key half][row]: maximum of the tile
    alignas(16) float alpha[2][kRows];      // the factors of the tile: the score rank's, copied to the value rank
    float fin[kRows];                       // value pair: 1 / l; -1: nothing visible
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

struct Batch {
    const int32_t* seq_lens;
    const int32_t* cu_q;
    int B, T, H, max_pages;
    int per;               // query tokens of a row tile: 128 / H
    // requests [cu_group[g], cu_group[g + 1]) have their first shared_lens[g] positions in common
    const int32_t* cu_group;
    const int32_t* shared_lens;
    int G;
    int units;             // numbers that the units lie within: T / (2 per) + G + 3
    int shift;             // 2 per = 1 << shift
};

__device__ __forceinline__ int token_at(const Batch& bt, int b) { return max(0, min(bt.T, __ldg(bt.cu_q + b))); }
// Lengths below 0 count as 0.
__device__ __forceinline__ int seq_len(const Batch& bt, int b) { return max(0, __ldg(bt.seq_lens + b)); }

// First request of span k: span 0 are the requests in front of all groups, k = 1 .. G group k - 1, G + 1 those behind.
__device__ __forceinline__ int span_begin(const Batch& bt, int k) {
    if (k <= 0) return 0;
    if (k > bt.G + 1 || bt.G == 0) return bt.B;
    return max(0, min(bt.B, __ldg(bt.cu_group + k - 1)));
}
// Positions of its shared prefix: whole pages, inside the table.
__device__ __forceinline__ int span_prefix(const Batch& bt, int k) {
    return k < 1 || k > bt.G ? 0 : max(0, min(bt.max_pages, __ldg(bt.shared_lens + k - 1) / kPage)) * kPage;
}
// Number of its first unit: the last one's is below the next span's.
__device__ __forceinline__ int span_unit(const Batch& bt, int k) { return (token_at(bt, span_begin(bt, k)) >> bt.shift) + k; }

struct Unit {
    int q0, nq;            // query tokens
    int prefix;            // positions of the shared prefix
    int b0;                // the request through whose row of the table it is read
    int requests, span_q0, span_nq;    // of the whole group
};

__device__ __forceinline__ Unit unit_of(const Batch& bt, int i) {
    int k = 0;                                                   // the last span whose numbers begin at or before i
    for (int hi = bt.G + 1; k < hi;) {
        const int mid = (k + hi + 1) >> 1;
        if (span_unit(bt, mid) <= i) k = mid; else hi = mid - 1;
    }
    const int b0 = span_begin(bt, k), b1 = max(b0, span_begin(bt, k + 1));
    const int q0 = token_at(bt, b0), nq = b1 > b0 ? max(0, token_at(bt, b1) - q0) : 0;
    const int64_t at = static_cast<int64_t>(i - span_unit(bt, k)) << bt.shift;
    Unit u{0, 0, span_prefix(bt, k), min(b0, bt.B - 1), b1 - b0, q0, nq};
    if (at >= 0 && at < nq) {
        u.q0 = q0 + static_cast<int>(at);
        u.nq = min(2 * bt.per, nq - static_cast<int>(at));
    }
    return u;
}

// The request of query token r, which is one of [b0, b1)'s: where all have as many tokens, the first guess.
__device__ __forceinline__ int request_of(const Batch& bt, const Unit& u, int r) {
    const int guess = u.b0 + min(u.requests - 1, static_cast<int>(__fdividef(static_cast<float>(r - u.span_q0) * u.requests, static_cast<float>(u.span_nq))));
    if (guess >= 0 && guess < bt.B && __ldg(bt.cu_q + guess) <= r && r < __ldg(bt.cu_q + guess + 1)) return guess;
    return row_request(bt.cu_q, bt.B, r);
}

// Keys that query token r, of request b, sees.
__device__ __forceinline__ int64_t sees_of(const Batch& bt, int b, int r) {
    const int q0 = token_at(bt, b), nq = max(0, token_at(bt, b + 1) - q0);
    return static_cast<int64_t>(seq_len(bt, b)) - nq + (r - q0) + 1;
}
// A query token of a unit: its request, the keys it sees of the prefix and behind it.
struct Token {
    int b, seen, own;
    bool cut;              // visible keys past the block table
};
// b: a request at or before the token's (the one of an earlier token of the unit).
__device__ __forceinline__ Token token_of(const Batch& bt, const Unit& u, int r, int b) {
    while (b + 1 < bt.B && __ldg(bt.cu_q + b + 1) <= r) ++b;
    const int64_t sees = sees_of(bt, b, r);
    const int64_t room = static_cast<int64_t>(bt.max_pages) * kPage - u.prefix;
    Token t;
    t.b = b;
    t.seen = static_cast<int>(max(static_cast<int64_t>(0), min(sees, static_cast<int64_t>(u.prefix))));
    t.own = static_cast<int>(max(static_cast<int64_t>(0), min(sees - u.prefix, room)));
    t.cut = sees - u.prefix > room;
    return t;
}
// A unit's prefix ends with the last page that one of its tokens sees the whole of: what lies behind that may not be there.
__device__ __forceinline__ int seen_prefix(const Unit& u, int64_t most) {
    return static_cast<int>(min(static_cast<int64_t>(u.prefix), max(static_cast<int64_t>(0), most) / kPage * kPage));
}
// Pages behind the prefix (of each request as many as its last token in the unit sees).
__device__ __forceinline__ int own_pages(const Batch& bt, Unit& u, bool& cut) {
    const int b0 = request_of(bt, u, u.q0);
    int64_t most = 0;
    for (int j = 0, b = b0; j < u.nq && most < u.prefix; ++j) {
        while (b + 1 < bt.B && __ldg(bt.cu_q + b + 1) <= u.q0 + j) ++b;
        most = max(most, sees_of(bt, b, u.q0 + j));
    }
    u.prefix = seen_prefix(u, most);
    Token t = token_of(bt, u, u.q0, b0);
    int pages = 0;
    cut = t.cut;
    for (int j = 1; j < u.nq; ++j) {
        const Token next = token_of(bt, u, u.q0 + j, t.b);
        if (next.b != t.b) pages += (t.own + kPage - 1) / kPage;
        t = next;
        cut |= t.cut;
    }
    return pages + (t.own + kPage - 1) / kPage;
}
// The same by a warp, a token a lane: lane j's token, the first of its request's pages among the unit's, how many (at the
// request's last token, else 0).  Returns all of the unit's pages.
__device__ __forceinline__ int unit_segments(const Batch& bt, Unit& u, Token& tok, int& seg_at, int& seg_pages) {
    const int lane = threadIdx.x & 31;
    tok = Token{-1, 0, 0, false};
    int b = 0, most = 0;
    if (lane < u.nq) {
        b = request_of(bt, u, u.q0 + lane);
        most = static_cast<int>(max(static_cast<int64_t>(0), min(sees_of(bt, b, u.q0 + lane), static_cast<int64_t>(u.prefix))));
    }
    u.prefix = seen_prefix(u, __reduce_max_sync(0xffffffffu, most));
    if (lane < u.nq) tok = token_of(bt, u, u.q0 + lane, b);
    const int next_b = __shfl_down_sync(0xffffffffu, tok.b, 1);
    seg_pages = lane < u.nq && (lane == u.nq - 1 || next_b != tok.b) ? (tok.own + kPage - 1) / kPage : 0;
    int upto = seg_pages;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    seg_at = u.prefix / kPage + upto - seg_pages;
    return u.prefix / kPage + __shfl_sync(0xffffffffu, upto, 31);
}
// Key tiles of a unit in the schedule: one that sees nothing counts as one.
__device__ __forceinline__ int schedule_tiles(int pages) { return max(1, (pages + 1) / 2); }

// A share's pieces, one unit after the other (a whole warp).
struct Walk {
    Batch bt;
    int i, left;           // unit, tiles left in the share
    Unit u;
    int pages, tiles;      // of the unit
    int t0, t1;
    bool whole, first;
    bool nothing;          // no piece at all
    bool inside;           // no token sees more than a part of the prefix's next page: what lies behind is all in that page
    int at, cost;          // where in the unit's length the share is; what of that comes in front of its tiles
    Token tok;             // lane j: token j's (see Piece)
    int seg_at, seg_pages;

    __device__ Walk(const Batch& batch, const Share& s) : bt(batch) {
        i = uniform(s.unit);
        at = uniform(s.at);
        cost = uniform(s.cost);
        left = uniform(s.left);
        first = true;
        u = unit_of(bt, i);
        set_piece();
    }
    __device__ void set_piece() {
        u.q0 = uniform(u.q0);
        u.nq = uniform(u.nq);
        u.prefix = uniform(u.prefix);
        const int common = u.prefix;
        pages = uniform(unit_segments(bt, u, tok, seg_at, seg_pages));
        inside = u.prefix < common;
        tiles = (pages + 1) / 2;
        // of the unit's length (what a change of units costs, then the tiles) from `at` on
        const int n = cost + schedule_tiles(pages);
        const int take = min(n - at, left);
        t0 = max(0, at - cost);
        whole = t0 == 0 && at + take == n;
        left -= take;
        t1 = min(max(0, at + take - cost), tiles);
        nothing = at + take <= cost;                             // the share ends before the first tile
    }
    // false: the share is done
    __device__ bool next() {
        if (left <= 0) return false;
        at = 0;
        first = false;
        do {
            if (++i >= bt.units) return false;
            u = unit_of(bt, i);
        } while (u.nq == 0);
        set_piece();
        return !nothing;
    }
};

// The pieces as the other warps read them.  One warp finds them for all: with that code inlined in every role, each role
// fetched its own copy at the first piece (5 prefixes, 32 heads: 98 -> 96.5 us; 32 requests of 16K keys, 128 heads: 120 -> 118.5).
struct Reader {
    Bars& bar;
    int per;
    uint32_t n = 0;        // pieces read
    bool late = false;     // a wait ran out
    int q0 = 0, nq = 0, prefix = 0, pages = 0, t0 = 0, t1 = 0;      // (no rows, if the first wait runs out)
    bool whole = false, first = false;

    __device__ Reader(Bars& b, int per_) : bar(b), per(per_) { load(); }
    __device__ const Piece& piece() const { return bar.piece[n % kPieces]; }
    __device__ bool load() {
        if (!ptx::mbar_wait(&bar.piece_full[n % kPieces], (n / kPieces) & 1u, ptx::wait_deadline())) late = true;
        late = __any_sync(0xffffffffu, late);
        if (late) return false;
        const Piece& p = piece();
        if (uniform(p.end) != 0) return false;
        q0 = uniform(p.q0);
        nq = uniform(p.nq);
        prefix = uniform(p.prefix);
        pages = uniform(p.pages);
        t0 = uniform(p.t0);
        t1 = uniform(p.t1);
        whole = uniform(p.whole) != 0;
        first = uniform(p.first) != 0;
        return true;
    }
    // false: the share is done
    __device__ bool next() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bar.piece_free[n % kPieces]);
        ++n;
        return load();
    }
    // Tokens of one rank's row tile
    __device__ int tokens(int side) const { return max(0, min(per, nq - side * per)); }
    // Page `at` of the unit's keys counts for tokens of one request only, not for all rows (a whole warp): the rows of other
    // tokens (word i: rows 32 i .. + 31), whose P there is 0, but 0 times an infinite or NaN value is not.
    __device__ bool others_rows(int at, int H, uint32_t (&off)[8]) const {
        if (at < prefix / kPage) return false;
        const Piece& p = piece();
        const int j = min(static_cast<int>(threadIdx.x & 31), kUnitTokens - 1);
        const bool sees = at >= p.at[j] && at - p.at[j] < (p.own[j] + kPage - 1) / kPage;
        const uint32_t all = (1u << nq) - 1u, mine = __ballot_sync(0xffffffffu, sees) & all;
        if (mine == all) return false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = 32 * i / H;                            // the token of row 32 i; of 16 rows each: two to a word
            const uint32_t a = (mine >> t) & 1u, b = H == 16 ? (mine >> (t + 1)) & 1u : a;
            off[i] = (a != 0u ? 0u : 0xffffu) | (b != 0u ? 0u : 0xffff0000u);
        }
        return true;
    }
    // Page `at` of the unit's keys: its entry in the block table, and how many of its rows count.
    __device__ int64_t page_entry(int max_pages, int at, int& valid) const {
        const Piece& p = piece();
        int64_t entry = static_cast<int64_t>(p.b0) * max_pages + at;
        valid = kPage;
#pragma unroll 1
        for (int j = 0; j < nq; ++j) {
            const int from = p.at[j], n_of = p.n[j];
            if (at >= from && at < from + n_of) {
                entry = static_cast<int64_t>(p.b[j]) * max_pages + prefix / kPage + (at - from);
                valid = min(kPage, p.own[j] - (at - from) * kPage);
            }
        }
        return entry;
    }
};

// The share of cluster c: lengths of all units in `sums` (shared), then one warp finds the start.
__device__ __forceinline__ void find_share(const Batch& bt, int c, int clusters, int* sums, Share& out, int32_t* err) {
    // few units: a warp each, a token a lane; many: a thread each, one token after the other
    bool cut = false;
    if (bt.units <= 64) {
        for (int i = threadIdx.x >> 5; i < bt.units; i += kThreads / 32) {
            Unit u = unit_of(bt, i);
            Token tok;
            int seg_at, seg_pages;
            const int pages = unit_segments(bt, u, tok, seg_at, seg_pages);
            cut |= tok.cut;
            if ((threadIdx.x & 31) == 0) sums[i] = u.nq > 0 ? schedule_tiles(pages) : 0;
        }
    } else {
        for (int i = threadIdx.x; i < bt.units; i += kThreads) {
            Unit u = unit_of(bt, i);
            bool c = false;
            const int own = u.nq > 0 ? own_pages(bt, u, c) : 0;
            sums[i] = u.nq > 0 ? schedule_tiles(u.prefix / kPage + own) : 0;
            cut |= c;
        }
    }
    if (cut && err != nullptr) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    if (err != nullptr) {
        for (int b = threadIdx.x; b < bt.B; b += kThreads)
            if (__ldg(bt.cu_q + b) < 0 || __ldg(bt.cu_q + b + 1) > bt.T) raise_error(err, DSA_DEVERR_INDEX_RANGE);
        for (int g = threadIdx.x; g < bt.G; g += kThreads)
            if (__ldg(bt.cu_group + g) < 0 || __ldg(bt.cu_group + g + 1) < __ldg(bt.cu_group + g) ||
                __ldg(bt.cu_group + g + 1) > bt.B || __ldg(bt.shared_lens + g) / kPage > bt.max_pages)
                raise_error(err, DSA_DEVERR_INDEX_RANGE);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int tiles = 0, some = 0;
        for (int i = lane; i < bt.units; i += 32) {
            tiles += sums[i];
            some += sums[i] > 0 ? 1 : 0;
        }
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        some = __reduce_add_sync(0xffffffffu, some);
        // a cluster that changes units gets fewer tiles (64 requests behind 32K: 119 -> 108 us); few tiles are cut as they are
        const int cost = tiles >= kLongShare * clusters ? kUnitCost : 0;
        const int total = tiles + some * cost;
        const int share = max((total + clusters - 1) / clusters, cost + kMinShare);
        const int64_t w0 = static_cast<int64_t>(c) * share;
        if (lane == 0) out.cost = cost;
        if (lane == 0) out.left = w0 < total ? static_cast<int>(min(static_cast<int64_t>(share), total - w0)) : 0;
        int carry = 0;
        for (int i0 = 0; i0 < bt.units && w0 < total; i0 += 32) {
            const int i = i0 + lane;
            const int own = i < bt.units && sums[i] > 0 ? sums[i] + cost : 0;
            int inc = own;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, w0 < carry + inc);
            if (hit != 0u) {
                if (lane == __ffs(hit) - 1) {
                    const int at = carry + inc - own;            // length before the unit
                    out.unit = i;
                    out.at = static_cast<int>(w0 - at);
                    out.first = (at + cost) / share;
                }
                break;
            }
            carry += __shfl_sync(0xffffffffu, inc, 31);
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
// Arrive on another CTA's barrier, with what this thread wrote before it ...
__device__ __forceinline__ void arrive_remote_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// ... or without ordering anything before it: used for buffers this thread has only read (the values are in registers).
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The pair's forms of the tensor-core instructions (every one of a kernel has to be of the same form).
__device__ __forceinline__ void umma2_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma2_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// ... into the accumulator's rows whose bits are not set in `off` (word i: rows 32 i .. + 31 of the pair's 256).
__device__ __forceinline__ void umma2_ss_rows(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, const uint32_t (&off)[8]) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]), "r"(off[5]),
        "r"(off[6]), "r"(off[7])
        : "memory");
}
// Arrive on the barrier at this offset in the CTAs of `mask` once the MMAs issued so far have completed.
__device__ __forceinline__ void umma2_commit(uint64_t* bar, uint32_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_addr(bar)),
        "h"(static_cast<uint16_t>(mask))
        : "memory");
}
__device__ __forceinline__ void tmem2_alloc(uint32_t* dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// TMA load into this CTA's shared memory, counted on a barrier of the pair's leader (its shared::cluster address).
__device__ __forceinline__ void tma2_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// What a cluster leaves for the combine kernel, for each rank of the pair: the split unit whose last piece it computed.
struct Meta {
    int64_t out_row;       // first output row (token * H)
    int rows;              // its rows; 0: none
    int first_cluster;
};

// The tensor maps: cache pages (64 rows, 8 rows and 1 row of 64 dims), queries, output, partial results.
struct Maps {
    CUtensorMap kv, kv8, kv1, q, out, part;
};

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(4, 1, 1)
dense_mla_shared_kernel(const __grid_constant__ Maps maps, const uint16_t* __restrict__ kv, int num_pages,
                        const int32_t* __restrict__ block_table, Batch bt, float scale, uint16_t* __restrict__ out,
                        float* __restrict__ lse_out, float* __restrict__ part_lse, Meta* __restrict__ meta, int slot_rows,
                        int32_t* err) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    unsigned char* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    unsigned char* ring = base;                                                   // key / value stages
    unsigned char* qrope = base + kKStages * kKStageBytes;                        // score pair: [128 rows][64 dims]
    unsigned char* ps = base + kPOffset;                                          // [4 pages][128 rows][64 keys]
    Bars& bar = *reinterpret_cast<Bars*>(base + kDataBytes);

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t cta = uniform(cluster_ctarank());
    const bool scores = cta < 2;
    const int side = static_cast<int>(cta & 1u);                 // which 128 rows of the unit
    const bool leader = side == 0;
    const uint32_t leader_cta = cta & 2u, both = scores ? 0x3u : 0xcu;
    const int cluster = blockIdx.x >> 2, clusters = gridDim.x >> 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(&bar.kv_full[s], 1);
            ptx::mbar_init(&bar.kv_empty[s], 1);
        }
        for (int s = 0; s < kQStages; ++s) {
            ptx::mbar_init(&bar.q_land[s], 1);
            ptx::mbar_init(&bar.q_read[s], 2);
        }
        ptx::mbar_init(&bar.lead_pass, 1);
        for (int i = 0; i < kPieces; ++i) {
            ptx::mbar_init(&bar.piece_full[i], 1);
            ptx::mbar_init(&bar.piece_free[i], kReaders);
        }
        bar.stop = 0;
        ptx::mbar_init(&bar.q_full, 16);
        for (int i = 0; i < kSBufs; ++i) {
            ptx::mbar_init(&bar.s_full[i], 1);
            ptx::mbar_init(&bar.s_read[i], 16);
        }
        for (int i = 0; i < kInfo; ++i) ptx::mbar_init(&bar.info[i], 1);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&bar.pair[i], 2);
        for (int i = 0; i < kPBufs; ++i) {
            ptx::mbar_init(&bar.p_free[i], 1);
            ptx::mbar_init(&bar.p_full[i], 1);
            ptx::mbar_init(&bar.p_peer[i], 1);
        }
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&bar.scaled[i], 8);
        for (int i = 0; i < kPvBars; ++i) ptx::mbar_init(&bar.pv_done[i], 1);
        ptx::mbar_init(&bar.o_free, 16);
        ptx::mbar_init(&bar.fin_full, 1);
        ptx::mbar_init(&bar.stage_lent, 1);
        ptx::mbar_init(&bar.stage_back, 8);
        ptx::mbar_init(&bar.fin_free, 8);
        ptx::fence_barrier_init();
    }
    ptx::griddep_wait();             // a programmatic dependent: what came before is complete
    find_share(bt, cluster, clusters, reinterpret_cast<int*>(ring), bar.share, cluster == 0 && cta == 0 ? err : nullptr);
    ptx::fence_proxy_async_smem();   // the schedule's scratch lies where copies will land
    cluster_sync_all();              // all CTAs' barriers exist before a peer signals or writes into them
    if (warp == kMmaWarp) tmem2_alloc(&bar.tmem_slot, 512);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = uniform(bar.tmem_slot);
    // limit of every wait, set anew every 256 tiles: a wait lasts a tile or so, the kernel may run for seconds
    uint64_t deadline = ptx::wait_deadline();
    bool timed_out = false;
    const bool work = uniform(bar.share.left) > 0;   // (its first unit may begin after the share's end)
    const uint32_t ring_addr = ptx::smem_addr(ring);
    const int pair_id = 2 * cluster + side;
    // workspace slot of a piece that is not a whole unit: 2 c for the one that starts share c but not its unit, else 2 c + 1
    auto piece_slot = [&](const Reader& w) { return 2 * static_cast<int64_t>(pair_id) + ((w.first && w.t0 > 0) ? 0 : 1); };
    if (threadIdx.x == 0 && !scores) meta[pair_id].rows = 0;

    if (work && warp == kTmaWarp) {
        // ---------------------------------------------------------------- TMA (all ranks)
        const uint32_t stages = scores ? kKStages : kVStages;
        Reader w(bar, bt.per);
        uint32_t s = 0, ph = 0, used = 0, u = 0;                     // stage, its phase, stages used so far, tiles
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
        const uint32_t full0 = map_to_rank(ptx::smem_addr(&bar.kv_full[0]), leader_cta);
        do {
            // the row tile's queries, 64 rows x 64 dims a stage (rows past its last one are other tokens', or zeros)
            if (scores && w.t0 < w.t1)
                for (int c = 0; c < kQStages && stage(); ++c) {
                    if (elect_one()) {
                        if (leader) ptx::mbar_arrive(&bar.kv_full[s]);   // no keys in it: the stage's phase passes first
                        ptx::mbar_arrive_expect_tx(&bar.q_land[c], kKStageBytes);
                        ptx::tma_load_3d(ring + s * kKStageBytes, &maps.q, &bar.q_land[c], (c >> 1) * 64, 0,
                                         (w.q0 + side * bt.per) * bt.H + (c & 1) * 64);
                    }
                    advance();
                }
            auto load_pages = [&](int t, int& valid) {               // page ids of 16 tiles from t on
                const int at = 2 * t + lane;
                const int64_t entry = w.page_entry(bt.max_pages, at, valid);
                return at < 2 * w.t1 && at < w.pages ? __ldg(block_table + entry) : -1;
            };
            int valid = 0, valid_next = 0;
            int page = -1, page_next = w.t0 < w.t1 ? load_pages(w.t0, valid_next) : -1;
            for (int t = w.t0; t < w.t1 && !timed_out; ++t, ++u) {
                const int tb = (t - w.t0) & 15;
                if (tb == 0) {
                    deadline = ptx::wait_deadline();
                    page = page_next;
                    valid = valid_next;
                    page_next = load_pages(t + 16, valid_next);
                }
                if (!scores && t + kAhead < w.t1) {
                    // the pages kAhead tiles further into L2, one a rank
                    const int src = 2 * (tb + kAhead) + side;
                    const int near = __shfl_sync(0xffffffffu, page, src & 31), far = __shfl_sync(0xffffffffu, page_next, src & 31);
                    const int pg = src < 32 ? near : far;
                    if (pg >= 0 && pg < num_pages) {
                        const unsigned char* p = reinterpret_cast<const unsigned char*>(kv + static_cast<int64_t>(pg) * (kPage * kLatentDim));
#pragma unroll
                        for (int j = 0; j < kPage * kLatentDim * 2 / 4096; ++j) prefetch_line(p + (j * 32 + lane) * 128);
                    }
                }
                int row[2], ok = 0, rows_of[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pg = __shfl_sync(0xffffffffu, page, 2 * tb + i);
                    const bool needed = 2 * t + i < w.pages;
                    const bool there = needed && pg >= 0 && pg < num_pages;
                    // a page that is not there: a box past the end reads zeros, and its keys are masked
                    row[i] = (there ? pg : num_pages) * kPage;
                    rows_of[i] = there ? __shfl_sync(0xffffffffu, valid, 2 * tb + i) : kPage;
                    ok |= there ? 1 << i : 0;
                    if (needed && !there && lane == 0 && cta == 0) raise_error(err, DSA_DEVERR_PAGE_RANGE);
                }
                if (scores) {
                    if (lane == 0) {
                        bar.tile_ok[u % kInfo] = ok;
                        ptx::mbar_arrive(&bar.info[u % kInfo]);
                    }
                    for (int c = 0; c < 9 && stage(); ++c) {
                        if (elect_one()) {
                            if (leader) ptx::mbar_arrive_expect_tx(&bar.kv_full[s], 2 * kKStageBytes);
                            tma2_load_3d(ring + s * kKStageBytes, &maps.kv, full0 + s * 8, c * 64, 0, side == 0 ? row[0] : row[1]);
                        }
                        advance();
                    }
                } else {
                    for (int i = 0; i < 4 && stage(); ++i) {         // page i / 2, of value dims 256 (i % 2) .. + 255 this rank's 128
                        const int r0 = i < 2 ? row[0] : row[1], n = i < 2 ? rows_of[0] : rows_of[1];
                        unsigned char* dst = ring + s * kVStageBytes;
                        const int d0 = (i & 1) * 256 + side * 128;
                        if (leader && elect_one()) ptx::mbar_arrive_expect_tx(&bar.kv_full[s], 2 * kVStageBytes);
                        __syncwarp();
                        if (n >= kPage) {
                            if (elect_one()) {
                                tma2_load_3d(dst, &maps.kv, full0 + s * 8, d0, 0, r0);
                                tma2_load_3d(dst + kPageChunk, &maps.kv, full0 + s * 8, d0 + 64, 0, r0);
                            }
                        } else {
                            // rows past the last visible position may hold anything: their P is 0, but 0 times NaN or
                            // infinity is not.  So only the rows that count are copied, by eights and one by one (boxes past the
                            // cache's end fill the others with zeros); lane j: rows 8 (j / 2) .. + 7 of 64 dims
                            if (lane < 16) {
                                unsigned char* at = dst + (lane & 1) * kPageChunk + (lane >> 1) * 1024;
                                const int first = (lane >> 1) * 8, dim = d0 + (lane & 1) * 64;
                                if (n >= first + 8 || n <= first) {
                                    tma2_load_3d(at, &maps.kv8, full0 + s * 8, dim, 0, n > first ? r0 + first : num_pages * kPage);
                                } else {
                                    for (int j = 0; j < 8; ++j)
                                        tma2_load_3d(at + j * 128, &maps.kv1, full0 + s * 8, dim, 0,
                                                     first + j < n ? r0 + first + j : num_pages * kPage);
                                }
                            }
                        }
                        advance();
                    }
                }
            }
            // value ranks: four stages for the row tile's output
            if (!scores && w.t0 < w.t1 && !timed_out) {
                for (int i = 0; i < kLent && stage(); ++i) {
                    if (elect_one()) {
                        if (leader) ptx::mbar_arrive(&bar.kv_full[s]);   // nothing to copy: the stage's phase passes
                        if (i == kLent - 1) ptx::mbar_arrive(&bar.stage_lent);
                    }
                    advance();
                }
            }
        } while (!timed_out && w.next());
        timed_out |= w.late;
        // copies still in flight land before the cluster may leave (bounded): the leader sees both ranks'
        if (leader)
            for (uint32_t j = used > stages ? used - stages : 0; j < used; ++j)
                if (!ptx::mbar_wait(&bar.kv_full[j % stages], (j / stages) & 1u, ptx::wait_deadline(20000000ull))) timed_out = true;
    } else if (work && warp == kMmaWarp && scores && leader) {
        // ---------------------------------------------------------------- MMA: S = Q K^T, for both ranks
        constexpr uint32_t idesc = ptx::instr_desc(1, 1, 2 * kRows, kKeys);
        const uint32_t pass_there = map_to_rank(ptx::smem_addr(&bar.lead_pass), cta + 1u);
        const uint64_t k_desc = desc_sw128(ring_addr, 16, 1024), qr_desc = desc_sw128(ptx::smem_addr(qrope), 16, 1024);
        // a wait that ran out only marks the step; the warp leaves at its end
        bool late = false;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) late = true;
        };
        Reader w(bar, bt.per);
        uint32_t u = 0, seg = 0, s = 0, ph = 0;
        do {
            if (w.t0 >= w.t1) continue;
            for (int c = 0; c < kQStages; ++c) {
                wait(&bar.q_read[c], seg & 1u);
                __syncwarp();
                if (elect_one()) ptx::mbar_arrive(&bar.kv_empty[s]);
                __syncwarp();
                if (++s == kKStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (elect_one()) arrive_remote_release(pass_there);
            __syncwarp();
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
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (c < 8) umma2_ts(d, tmem + c * 32 + kk * 8, so + kk * 2, idesc, (c | kk) != 0 ? 1u : 0u);
                            else umma2_ss(d, qr_desc + kk * 2, so + kk * 2, idesc, 1u);
                        }
                        umma2_commit(&bar.kv_empty[s], both);
                        if (c == 8) umma2_commit(&bar.s_full[sb], both);
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
        if (late || w.late) timed_out = true;
    } else if (work && warp == kMmaWarp && scores) {
        // ---------------------------------------------------------------- the other score rank: its query stages given back
        Reader w(bar, bt.per);
        uint32_t seg = 0, s = 0;
        do {
            if (w.t0 >= w.t1) continue;
            deadline = ptx::wait_deadline();
            if (!ptx::mbar_wait(&bar.lead_pass, seg & 1u, deadline)) timed_out = true;
            timed_out = __any_sync(0xffffffffu, timed_out);
            for (int c = 0; c < kQStages && !timed_out; ++c) {
                if (!ptx::mbar_wait(&bar.q_read[c], seg & 1u, deadline)) timed_out = true;
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (lane == 0) ptx::mbar_arrive(&bar.kv_empty[s]);
                s = (s + 1) % kKStages;
            }
            ++seg;
            s = (s + 9u * static_cast<uint32_t>(w.t1 - w.t0)) % kKStages;
        } while (!timed_out && w.next());
        timed_out |= w.late;
    } else if (work && warp == kMmaWarp && leader) {
        // ---------------------------------------------------------------- MMA: O += P V, for both ranks
        constexpr uint32_t idesc = ptx::instr_desc(1, 1, 2 * kRows, 256) | (1u << 16);   // B MN-major
        const uint32_t pass_there = map_to_rank(ptx::smem_addr(&bar.lead_pass), cta + 1u);
        const uint64_t v_desc = desc_sw128(ring_addr, kPageChunk, 1024), p_desc = desc_sw128(ptx::smem_addr(ps), 16, 1024);
        bool late = false;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) late = true;
        };
        Reader w(bar, bt.per);
        uint32_t u = 0, seg = 0, s = 0, ph = 0;
        do {
            if (w.t0 >= w.t1) continue;
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                bool part = false;
                uint32_t off[8] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {                        // page i / 2, value dims 256 (i % 2) .. + 255
                    const uint32_t pb = 2 * (u & 1u) + (i >> 1);
                    // a page of one request's: into its rows alone (O begins with zeros where it is the piece's first page)
                    if ((i & 1) == 0) part = w.others_rows(2 * t + (i >> 1), bt.H, off);
                    wait(&bar.kv_full[s], ph);
                    if ((i & 1) == 0) {
                        wait(&bar.p_full[pb], (u >> 1) & 1u);
                        wait(&bar.p_peer[pb], (u >> 1) & 1u);
                    }
                    if (i == 0) {
                        if (t == w.t0 && seg > 0) wait(&bar.o_free, (seg - 1) & 1u);
                        wait(&bar.scaled[u & 1], (u >> 1) & 1u);
                    }
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t vb = v_desc + s * (kVStageBytes / 16);
                        const uint64_t pd = p_desc + pb * (kPBytes / 16);
                        if (part) {
#pragma unroll
                            for (int ks = 0; ks < kPage / 16; ++ks)
                                umma2_ss_rows(tmem + (i & 1) * 256, pd + ks * 2, vb + ks * 128, idesc, off);
                        } else {
#pragma unroll
                            for (int ks = 0; ks < kPage / 16; ++ks)
                                umma2_ss(tmem + (i & 1) * 256, pd + ks * 2, vb + ks * 128, idesc, (t > w.t0 || i >= 2 || ks != 0) ? 1u : 0u);
                        }
                        umma2_commit(&bar.kv_empty[s], both);
                        if ((i & 1) == 1) umma2_commit(&bar.p_free[pb], 0x3u);
                        if (i == 3) umma2_commit(&bar.pv_done[u % kPvBars], both);
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
            __syncwarp();
            if (elect_one()) arrive_remote_release(pass_there);
            for (int i = 0; i < kLent; ++i) {
                __syncwarp();
                if (elect_one()) ptx::mbar_arrive(&bar.kv_empty[s]);
                if (++s == kVStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            ++seg;
        } while (!__any_sync(0xffffffffu, late) && w.next());
        if (late || w.late) timed_out = true;
    } else if (work && warp == kMmaWarp) {
        // ---------------------------------------------------------------- the other value rank: its P for the leader
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) timed_out = true;
        };
        const uint32_t there = map_to_rank(ptx::smem_addr(&bar.p_peer[0]), leader_cta);
        Reader w(bar, bt.per);
        uint32_t u = 0, seg = 0, s = 0;
        do {
            if (w.t0 >= w.t1) continue;
            for (int t = w.t0; t < w.t1 && !timed_out; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                const uint32_t pb = 2 * (u & 1u);
                wait(&bar.p_full[pb], (u >> 1) & 1u);
                wait(&bar.scaled[u & 1], (u >> 1) & 1u);
                ptx::tc_fence_after_sync();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_remote_release(there + pb * 8);
                wait(&bar.p_full[pb + 1], (u >> 1) & 1u);
                __syncwarp();
                if (lane == 0) arrive_remote_release(there + (pb + 1) * 8);
                timed_out = __any_sync(0xffffffffu, timed_out);
            }
            if (timed_out) break;
            s = (s + 4u * static_cast<uint32_t>(w.t1 - w.t0)) % kVStages;
            wait(&bar.lead_pass, seg & 1u);
            wait(&bar.stage_back, seg & 1u);
            timed_out = __any_sync(0xffffffffu, timed_out);
            for (int i = 0; i < kLent; ++i) {
                if (lane == 0) ptx::mbar_arrive(&bar.kv_empty[s]);
                s = (s + 1) % kVStages;
            }
            ++seg;
        } while (!timed_out && w.next());
        timed_out |= w.late;
    } else if (work && warp < kTmaWarp && scores) {
        // ---------------------------------------------------------------- softmax (score pair)
        const int quad = warp & 3, kh = warp >> 2;
        const int row = quad * 32 + lane;                            // query row of the row tile = tensor-memory lane
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const float cs = scale * kLog2e;
        const uint64_t cs2 = f32x2(cs, cs);
        const int token = side * bt.per + row / bt.H;                // of the unit
        const uint32_t p_row = row * 128, p_swz = row & 7;           // the row's place in a P buffer
        // this warp's 32 rows of a P buffer, and their factors, here and in the value rank
        const uint32_t value_cta = 2u + static_cast<uint32_t>(side);
        const uint32_t p_here = ptx::smem_addr(ps) + quad * 4096, p_there = map_to_rank(p_here, value_cta);
        const uint32_t a_here = ptx::smem_addr(&bar.alpha[0][quad * 32]), a_there = map_to_rank(a_here, value_cta);
        const uint32_t full_there = map_to_rank(ptx::smem_addr(&bar.p_full[0]), value_cta);
        const uint32_t read_there = map_to_rank(ptx::smem_addr(&bar.s_read[0]), leader_cta);
        const uint32_t q_there = map_to_rank(ptx::smem_addr(&bar.q_full), leader_cta);
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) timed_out = true;
        };
        uint32_t u = 0, seg = 0, meets = 0, used = 0;                // meets: uses of the pair barrier; used: ring stages
        Reader w(bar, bt.per);
        do {
            const int live = w.tokens(side) * bt.H;
            const bool quad_live = quad * 32 < live;
            // Rows behind the last one are other requests' queries, stale P and its products: nothing reads what comes
            // of them, but zeros there let the tensor cores idle, and a long call runs at the power limit
            const bool row_live = row < live;
            // the row's keys: [0, seen) of the prefix's pages, [lo, hi) of those behind
            const Piece& piece = w.piece();
            int seen = piece.seen[token];
            const int lo = piece.at[token] * kPage, own = piece.own[token];
            const int hi = row_live ? lo + own : lo;
            if (!row_live) seen = 0;
            float m_run = -INFINITY, l_run = 0.0f;
            if (w.t0 < w.t1) {
                // the row tile's queries out of the ring: value chunks into tensor memory, the rope chunk into its
                // place; even chunks by the warps of page 0, odd ones by those of page 1.  (The score MMAs
                // before are complete: their s_full has been waited for.  Warps without live rows have not passed a
                // fence since, and the stores to come may not move ahead of that wait.)
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < 9; ++c) {
                    if ((c & 1) == kh) {
                        const int qs = 2 * c + (quad >> 1);          // this warp's 64 rows
                        const uint32_t st = (used + qs) % kKStages;
                        wait(&bar.q_land[qs], seg & 1u);
                        const unsigned char* src = ring + st * kKStageBytes + (p_row & 8191u);
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
                        if (lane == 0) ptx::mbar_arrive(&bar.q_read[qs]);
                    }
                }
                // (the last two chunk halves' stages are read by the warps of page 0 alone)
                used += kQStages;
                tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_remote_release(q_there);
            }
            used += 9u * static_cast<uint32_t>(max(0, w.t1 - w.t0));
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                const uint32_t sb = u % kSBufs, pb = 2 * (u & 1u) + kh;
                wait(&bar.s_full[sb], (u / kSBufs) & 1u);
                if (quad_live) {
                    wait(&bar.info[u % kInfo], (u / kInfo) & 1u);
                    __syncwarp();
                    ptx::tc_fence_after_sync();
                    uint32_t v[2][32];
                    const uint32_t sa = tmem + lane_base + kColS + sb * kKeys + kh * kPage;
                    ptx::tmem_ld_32x32b_x32(sa, v[0]);
                    ptx::tmem_ld_32x32b_x32(sa + 32, v[1]);
                    const int at = t * kKeys + kh * kPage;           // the page's first position in the unit's keys
                    const bool behind = at >= w.prefix;
                    const int from = behind ? lo - at : 0;           // the row's: [from, lim)
                    const int lim = ((bar.tile_ok[u % kInfo] >> kh) & 1) ? (behind ? hi : seen) - at : 0;
                    ptx::tmem_wait_ld();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_remote(read_there + sb * 8);
                    if (lim < kPage || from > 0) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e >= lim || e < from) v[e >> 5][e & 31] = 0xff800000u;   // -inf
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
                    arrive_remote(read_there + sb * 8);
                }
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
            }
            if (timed_out) break;
            // ---- 1 / l to the value rank; the log-sum-exp (log2 units for a part)
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
                        st_async_f32(map_to_rank(ptx::smem_addr(&bar.fin[row]), value_cta), l_tot == 0.0f ? -1.0f : 1.0f / l_tot,
                                     map_to_rank(ptx::smem_addr(&bar.fin_full), value_cta));
                }
                if (kh == 0 && row < live) {
                    const float lse2 = l_tot == 0.0f ? -INFINITY : m_run * cs + log2f(l_tot);
                    if (!w.whole) part_lse[piece_slot(w) * slot_rows + row] = lse2;
                    else if (lse_out != nullptr) lse_out[static_cast<int64_t>(w.q0 + side * bt.per) * bt.H + row] = lse2 * kLn2;
                }
            }
            if (w.t0 < w.t1) ++seg;
        } while (w.next());
        timed_out |= w.late;
        // the value pair's last signals land here before this CTA may finish
        for (uint32_t j = 2 * u > kPBufs ? 2 * u - kPBufs : 0; j < 2 * u && !timed_out; ++j)
            wait(&bar.p_free[j % kPBufs], (j / kPBufs) & 1u);
    } else if (work && warp < kTmaWarp) {
        // ---------------------------------------------------------------- rescaling, output (value pair)
        const int quad = warp & 3, dh = warp >> 2;                   // rows 32 quad .. + 31, output dims 256 dh .. + 255
        const int row = quad * 32 + lane;
        const uint32_t o_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + dh * 256;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (!ptx::mbar_wait(b, parity, deadline)) timed_out = true;
        };
        uint32_t u = 0, seg = 0, used = 0;                           // used: ring stages before this row tile
        uint32_t clean = 0;                                          // bit i: this row group's P is zero in buffers 2 i and 2 i + 1
        const uint32_t free_there = map_to_rank(ptx::smem_addr(&bar.o_free), leader_cta);
        const uint32_t fin_free_there = map_to_rank(ptx::smem_addr(&bar.fin_free), static_cast<uint32_t>(side));
        Reader w(bar, bt.per);
        do {
            const int live = w.tokens(side) * bt.H;
            const int64_t out_row = static_cast<int64_t>(w.q0 + side * bt.per) * bt.H;
            const bool quad_live = quad * 32 < live, has_tiles = w.t0 < w.t1;
            const uint32_t quads = static_cast<uint32_t>((live + 31) / 32);
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                if ((u & 255u) == 0u) deadline = ptx::wait_deadline();
                const uint32_t pb = 2 * (u & 1u), pph = (u >> 1) & 1u;
                // a row tile without rows gets no P that would wait for the buffers' products to complete: wait here
                if (live == 0 && u >= 2) wait(&bar.pv_done[(u - 2) % kPvBars], ((u - 2) / kPvBars) & 1u);
                if (threadIdx.x == 0) {
                    // the second buffer's previous phase is over once its P V is: this warp has not waited for it
                    if (u >= 2) wait(&bar.p_full[pb + 1], pph ^ 1u);
                    ptx::mbar_arrive_expect_tx(&bar.p_full[pb], quads * (kPBytes / 4 + 32 * 4));
                    ptx::mbar_arrive_expect_tx(&bar.p_full[pb + 1], quads * (kPBytes / 4));
                }
                __syncwarp();
                if (t == w.t0 && quad_live) {
                    // the first page goes into one request's rows alone: the others begin with zeros
                    uint32_t off[8];
                    if (w.others_rows(2 * t, bt.H, off)) {
                        const uint32_t zero[32] = {};
#pragma unroll 1
                        for (int cc = 0; cc < 256; cc += 32) tmem_st_x32(o_addr + cc, zero);
                        tmem_wait_st();
                        ptx::tc_fence_before_sync();
                    }
                }
                wait(&bar.p_full[pb], pph);
                if (quad_live) {
                    clean &= ~(1u << (u & 1u));
                } else if (((clean >> (u & 1u)) & 1u) == 0u) {
                    // no P comes for these rows.  Only this tile's buffers: the score rank writes into them again when its
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
                // when the score rank learns that it may write the next ones
                hidden = __ballot_sync(0xffffffffu, inv < 0.0f);
                __syncwarp();
                if (lane == 0) arrive_remote(fin_free_there);
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
                const int64_t row0 = w.whole ? out_row : piece_slot(w) * slot_rows;
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
                    unsigned char* st = ring + ((used + 2 * buf + (warp >> 2)) % kVStages) * kVStageBytes + (warp & 3) * 4096;
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
                                tma_store_3d(w.whole ? &maps.out : &maps.part, st + h * 2048, dh * 256 + cc, 0,
                                             static_cast<int>(row0) + quad * 32 + 16 * h);
                        bulk_commit();
                    }
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    arrive_remote(free_there);
                    bulk_wait_read<0>();
                    ptx::mbar_arrive(&bar.stage_back);
                }
                used += kLent;
                ++seg;
            } else if (quad_live) {                                  // sees nothing: zeros
                for (int r = quad * 32; r < min(live, quad * 32 + 32); ++r)
                    *reinterpret_cast<uint4*>(out + (out_row + r) * kValueDim + dh * 256 + lane * 8) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            // the last piece of a split unit: the combine kernel finds it here
            if (threadIdx.x == 0 && w.first && w.t0 > 0 && w.t1 == (w.pages + 1) / 2 && live > 0)
                meta[pair_id] = Meta{out_row, live, bar.share.first};
        } while (w.next());
        timed_out |= w.late;
        if (lane == 0) bulk_wait_all();                              // written before the CTA leaves
    }
    if (work && warp == kWalkWarp) {
        // ---------------------------------------------------------------- the pieces, for all other warps
        Walk w(bt, bar.share);
        bool more = true;
        for (uint32_t n = 0;; ++n) {
            const uint32_t i = n % kPieces;
            // (a piece may take long: the others' waits are limited, and tell when one has run out)
            bool free = n < kPieces;
            for (int tries = 0; tries < 64 && !free && *static_cast<volatile int*>(&bar.stop) == 0; ++tries)
                free = ptx::mbar_wait(&bar.piece_free[i], ((n / kPieces) & 1u) ^ 1u, ptx::wait_deadline());
            if (!__all_sync(0xffffffffu, free)) {
                timed_out = true;
                break;
            }
            Piece& p = bar.piece[i];
            if (lane < kUnitTokens) {
                p.b[lane] = w.inside ? w.u.b0 : w.tok.b;
                p.at[lane] = w.seg_at;
                p.n[lane] = w.seg_pages;
                p.seen[lane] = w.tok.seen;
                p.own[lane] = w.tok.own;
            }
            if (lane == 0) {
                p.q0 = w.u.q0;
                p.nq = w.u.nq;
                p.prefix = w.u.prefix;
                p.b0 = w.u.b0;
                p.pages = w.pages;
                p.t0 = w.t0;
                p.t1 = w.t1;
                p.whole = w.whole;
                p.first = w.first;
                p.end = !more;
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar.piece_full[i]);
            if (!more) break;
            more = w.next();
        }
    }
    if (timed_out) {
        raise_error(err, DSA_DEVERR_TIMEOUT);
        *static_cast<volatile int*>(&bar.stop) = 1;
    }
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before_sync();
    cluster_sync_all();   // the pair's products are done with both tensor memories
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        tmem2_dealloc(tmem, 512);
    }
    cluster_sync_all();   // no CTA leaves while a peer may still signal or write into it
}

// Joins the pieces of the split units: those of a unit lie in slot 2 c0 + 1 of its first cluster's and 2 c of the
// following clusters' pairs of slots, each rank's rows for themselves.
__global__ void __launch_bounds__(kJoinThreads)
dense_mla_shared_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                const Meta* __restrict__ meta, int pairs, int slot_rows, uint16_t* __restrict__ out,
                                float* __restrict__ lse_out) {
    ptx::griddep_wait();
    join_listed(part_o, part_lse, pairs, slot_rows, out, lse_out, [&](int p) {
        const Meta m = meta[p];
        return JoinTask{m.out_row, m.rows, (p >> 1) - m.first_cluster + 1, 2 * (2 * m.first_cluster + (p & 1)), 4};
    });
}

// Clusters of four CTAs that the device holds at once (a GPC whose number of SMs is not a multiple of four leaves some
// over: 36 on a GPU of 152 SMs); asked once a device.
int shared_clusters() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max(4, device_sm_count() / 4 * 4)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, dense_mla_shared_kernel, &cfg) != cudaSuccess) return 0;
    n = std::min(n, device_sm_count() / 4);
    if (dev < 64 && n > 0) known[dev].store(n, std::memory_order_relaxed);
    return n;
}
// The workspace's size must not depend on what is asked of the device: pairs of slots for every cluster there could be.
int slot_pairs() { return std::max(1, device_sm_count() / 4) * 2; }
int shared_slot_rows(int64_t T, int64_t H) { return static_cast<int>(std::min<int64_t>(kRows, T * H)); }

}  // namespace
}  // namespace dsa

extern "C" size_t dsa_dense_mla_decode_shared_workspace_size(int32_t T, int32_t H) {
    using namespace dsa;
    if (T <= 0 || H <= 0) return 0;
    const size_t p = static_cast<size_t>(slot_pairs()), rows = static_cast<size_t>(shared_slot_rows(T, H));
    return p * sizeof(Meta) + 2 * p * rows * (kValueDim + 1) * sizeof(float);
}

extern "C" dsa_status dsa_dense_mla_decode_shared(const void* q_bf16, const void* kv_pool, int64_t num_pages,
                                                  const int32_t* block_table, int32_t max_pages,
                                                  const int32_t* seq_lens, const int32_t* cu_q, int32_t B, int32_t T,
                                                  int32_t H, const int32_t* cu_group, const int32_t* shared_lens,
                                                  int32_t G, float scale, void* out_bf16, float* lse, void* workspace,
                                                  size_t workspace_bytes, int32_t* dev_err, void* stream) {
    using namespace dsa;
    if (H != 16 && H != 32 && H != 64 && H != 128) return DSA_ERR_UNSUPPORTED;
    if (T < 0 || B < 0 || G < 0 || max_pages < 0 || num_pages < 0) return DSA_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return DSA_OK;
    if (num_pages < 1 || max_pages < 1) return DSA_ERR_INVALID_ARG;
    if (!q_bf16 || !kv_pool || !block_table || !seq_lens || !cu_q || !out_bf16) return DSA_ERR_INVALID_ARG;
    if (G > 0 && (!cu_group || !shared_lens)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_bf16) || !aligned16(kv_pool) || !aligned16(out_bf16)) return DSA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !(scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    if ((num_pages + 1) * kPage >= 0x7fffffffLL || static_cast<int64_t>(max_pages) * kPage >= 0x7fffffffLL || B > kMaxRequests ||
        G > kMaxGroups)
        return DSA_ERR_UNSUPPORTED;
    // one list of all units lies in shared memory; key tiles are counted in 32 bits, and a unit has up to 16 requests'
    if (static_cast<int64_t>(T) * H > static_cast<int64_t>(kMaxUnits) * 2 * kRows || static_cast<int64_t>(T) * max_pages >= 0x3fffffffLL)
        return DSA_ERR_UNSUPPORTED;
    // and so are the positions of a unit: the prefix and the own pages of all its requests, rounded up to a tile
    const int64_t unit_requests = std::min<int64_t>(std::min(T, B), 2 * kRows / H);
    if (unit_requests * max_pages * kPage >= 0x7fffffffLL - kKeys) return DSA_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < dsa_dense_mla_decode_shared_workspace_size(T, H))
        return DSA_ERR_INVALID_ARG;
    auto encode = attn::tensor_map_encoder();
    if (encode == nullptr) return DSA_ERR_CUDA;
    const int per = kRows / H, pairs = slot_pairs(), slot_rows = shared_slot_rows(T, H);
    const Batch bt{seq_lens, cu_q, B, T, H, max_pages, per, cu_group, shared_lens, G, T / (2 * per) + G + 3, H == 16 ? 4 : (H == 32 ? 3 : (H == 64 ? 2 : 1))};
    Meta* meta = static_cast<Meta*>(workspace);
    float* part_o = reinterpret_cast<float*>(meta + pairs);
    float* part_lse = part_o + static_cast<size_t>(2) * pairs * slot_rows * kValueDim;
    const uint64_t rows = static_cast<uint64_t>(T) * H, kv_rows = static_cast<uint64_t>(num_pages) * kPage;
    Maps maps;
    if (!attn::encode_bf16_3d(encode, &maps.kv, kv_pool, kLatentDim, 1, kv_rows, kLatentDim, kLatentDim, 64, kPage) ||
        !attn::encode_bf16_3d(encode, &maps.kv8, kv_pool, kLatentDim, 1, kv_rows, kLatentDim, kLatentDim, 64, 8) ||
        !attn::encode_bf16_3d(encode, &maps.kv1, kv_pool, kLatentDim, 1, kv_rows, kLatentDim, kLatentDim, 64, 1) ||
        !attn::encode_bf16_3d(encode, &maps.q, q_bf16, kLatentDim, 1, rows, kLatentDim, kLatentDim, 64, 64) ||
        !attn::encode_bf16_3d(encode, &maps.out, out_bf16, kValueDim, 1, rows, kValueDim, kValueDim, 64, 16) ||
        !attn::encode_f32_rows(encode, &maps.part, part_o, kValueDim, static_cast<uint64_t>(2) * pairs * slot_rows, 32, 16))
        return DSA_ERR_CUDA;
    if (cudaFuncSetAttribute(dense_mla_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess)
        return DSA_ERR_CUDA;
    const int clusters = shared_clusters();
    if (clusters < 1) return DSA_ERR_CUDA;
    // both kernels are programmatic dependents: scheduled as the CTAs of the one before end, they wait for all of it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4 * clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dense_mla_shared_kernel, maps, static_cast<const uint16_t*>(kv_pool),
                           static_cast<int>(num_pages), block_table, bt, scale, static_cast<uint16_t*>(out_bf16), lse,
                           part_lse, meta, slot_rows, dev_err) != cudaSuccess)
        return DSA_ERR_CUDA;
    cfg.gridDim = dim3(4 * clusters * kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, dense_mla_shared_combine_kernel, static_cast<const float*>(part_o),
                           static_cast<const float*>(part_lse), static_cast<const Meta*>(meta), 2 * clusters, slot_rows,
                           static_cast<uint16_t*>(out_bf16), lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}
