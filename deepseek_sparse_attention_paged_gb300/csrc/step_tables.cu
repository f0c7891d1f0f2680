// step_tables.cu -- block table, slot mapping, positions and row offsets of a step from the requests'
// lengths, with the pages that the step takes from and gives back to a free stack.
//
// Position p of request b lies in slot table[b][p / 64] * 64 + p % 64.
//
// Three prefix sums over the requests (new tokens, pages to take, pages given back) say everything: where a
// request's rows begin, which pages of the stack it gets, where its own go.  A page of the stack is found by
// its rank from the top; what is given back in the same call lies on top of it and is read from the tables
// of the requests that end, never from the part of the stack that this call writes.  So no CTA needs
// another's writes: each forms the sums for itself and takes its share of tokens and requests.
//
// Bound by latency: launch, lengths, sums, table, slots (a decode step moves a few KB).  Measured in a captured graph: one
// request 3.5 us, 500 with drafts 7.1 us, 48 prompts 5.5 us.
#include <algorithm>

#include "dsa_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kTabMaxRequests = 16384;          // three prefix sums in shared memory: 192 KB

struct StepTables {
    const int32_t *cached, *q_lens, *counts, *keep;
    int32_t* table;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t *seq_lens, *counts_out, *free_count_out, *cu_q;
    int64_t *positions, *slots;
    int B, T, max_pages, num_pages;
    int32_t* err;
};

// Exclusive prefix of v over the block's threads; `total` is the block's sum.  Sums saturate at `cap`
// (adding with saturation is associative for numbers >= 0).
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t cap, uint32_t* warp_sums, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc = min(cap, inc + o);
    }
    uint32_t exc = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) exc = 0;
    __syncthreads();                             // the sums of the call before have been read
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
    for (int w = 0; w < kTabWarps; ++w) {
        if (w == warp) before = total;
        total = min(cap, total + warp_sums[w]);
    }
    return min(cap, before + exc);
}

// Pages of request b that count (inside its row of the table).
__device__ __forceinline__ int mapped(const StepTables& s, int b) { return max(0, min(s.max_pages, __ldg(s.counts + b))); }
// Those of its pages that stay when it ends.
__device__ __forceinline__ int kept(const StepTables& s, int b, int c) {
    return s.keep != nullptr ? max(0, min(c, __ldg(s.keep + b))) : 0;
}

__global__ void __launch_bounds__(kTabThreads) step_tables_kernel(const StepTables s) {
    extern __shared__ uint32_t sums[];
    __shared__ uint32_t warp_sums[kTabWarps];
    uint32_t* cu = sums;                         // [B + 1] each: rows, pages taken, pages given back, before request b
    uint32_t* taken = cu + s.B + 1;
    uint32_t* given = taken + s.B + 1;
    ptx::griddep_wait();                         // a programmatic dependent: what came before is complete
    const int tid = threadIdx.x;
    const int per = (s.B + kTabThreads - 1) / kTabThreads;
    const int b0 = min(s.B, tid * per), b1 = min(s.B, b0 + per);
    const int have0 = max(0, min(s.num_pages, __ldg(s.free_count)));
    int bad = 0;
    // ---- the three prefix sums
    const uint32_t rows = static_cast<uint32_t>(s.T);
    uint32_t sum = 0, total;
    for (int b = b0; b < b1; ++b) sum = min(rows, sum + min(rows, static_cast<uint32_t>(max(0, __ldg(s.q_lens + b)))));
    uint32_t at = block_exclusive(sum, rows, warp_sums, total);
    if (tid == 0) cu[s.B] = total;
    for (int b = b0; b < b1; ++b) {
        cu[b] = at;
        const uint32_t n = static_cast<uint32_t>(max(0, __ldg(s.q_lens + b))), room = rows - at;
        if (n > room) bad |= DSA_DEVERR_INDEX_RANGE;
        at += min(n, room);
    }
    __syncthreads();
    uint32_t take = 0, give = 0;
    for (int b = b0; b < b1; ++b) {
        const int c = mapped(s, b);
        uint32_t t = 0, g = 0;
        if (__ldg(s.q_lens + b) < 0) {
            g = static_cast<uint32_t>(c - kept(s, b, c));
        } else {
            const int64_t len = static_cast<int64_t>(max(0, __ldg(s.cached + b))) + (cu[b + 1] - cu[b]);
            const int64_t need = (len + kPage - 1) / kPage;
            if (need > s.max_pages) bad |= DSA_DEVERR_INDEX_RANGE;
            t = static_cast<uint32_t>(max(0, static_cast<int>(min(need, static_cast<int64_t>(s.max_pages))) - c));
        }
        taken[b] = take;                         // before the request, within this thread's share
        given[b] = give;
        take += t;
        give += g;
    }
    uint32_t n_take, n_give;
    const uint32_t take0 = block_exclusive(take, 0x7fffffffu, warp_sums, n_take);
    const uint32_t give0 = block_exclusive(give, 0x7fffffffu, warp_sums, n_give);
    for (int b = b0; b < b1; ++b) {
        taken[b] += take0;
        given[b] += give0;
    }
    if (tid == 0) {
        taken[s.B] = n_take;
        given[s.B] = n_give;
    }
    __syncthreads();
    // pages on the stack once what ends has given its own back; a stack that overflows keeps what fits
    const int have = static_cast<int>(min(static_cast<int64_t>(have0) + n_give, static_cast<int64_t>(s.num_pages)));
    if (static_cast<int64_t>(have0) + n_give > s.num_pages) bad |= DSA_DEVERR_INDEX_RANGE;

    // The last request whose sum is at most x: it has x's row or page, as those behind with the same sum have none.
    auto owner = [&](const uint32_t* before, uint32_t x) {
        int lo = 0, hi = s.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= x) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    // The page of this rank from the top; -1: the stack is empty, or the entry is no page.
    auto page_of = [&](uint32_t rank) {
        if (rank >= static_cast<uint32_t>(have)) {
            bad |= DSA_DEVERR_NO_PAGE;
            return -1;
        }
        const int i = have - 1 - static_cast<int>(rank);
        int page;
        if (i < have0) {
            page = s.free_pages[i];
        } else {                                 // given back in this call
            const uint32_t j = static_cast<uint32_t>(i - have0);
            const int lo = owner(given, j), c = mapped(s, lo);
            page = s.table[static_cast<int64_t>(lo) * s.max_pages + kept(s, lo, c) + (j - given[lo])];
        }
        if (page < 0 || page >= s.num_pages) {
            bad |= DSA_DEVERR_PAGE_RANGE;
            return -1;
        }
        return page;
    };

    // ---- positions and slots, a row a thread
    const int used = static_cast<int>(cu[s.B]);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kTabThreads + tid; r < s.T; r += static_cast<int64_t>(gridDim.x) * kTabThreads) {
        int64_t pos = 0, slot = -1;
        if (r < used) {
            const int lo = owner(cu, static_cast<uint32_t>(r));
            pos = static_cast<int64_t>(max(0, __ldg(s.cached + lo))) + (r - cu[lo]);
            const int64_t p = pos / kPage;
            const int c = mapped(s, lo);
            if (p < s.max_pages) {
                int page;
                if (p < c) {
                    page = s.table[static_cast<int64_t>(lo) * s.max_pages + p];
                    if (page < 0 || page >= s.num_pages) {
                        bad |= DSA_DEVERR_PAGE_RANGE;
                        page = -1;
                    }
                } else {
                    page = page_of(taken[lo] + static_cast<uint32_t>(p - c));
                }
                if (page >= 0) slot = static_cast<int64_t>(page) * kPage + pos % kPage;
            }
        }
        s.positions[r] = pos;
        s.slots[r] = slot;
    }
    // ---- pages taken and given back, a page a thread (a warp a request would go over a long one's pages in turn: 40 of
    // 500 requests that end with up to 1000 pages 8.5 -> 7.0 us)
    const uint32_t first = blockIdx.x * kTabThreads + tid, stride = gridDim.x * kTabThreads;
    for (uint32_t i = first; i < n_take; i += stride) {
        const int b = owner(taken, i);
        s.table[static_cast<int64_t>(b) * s.max_pages + mapped(s, b) + (i - taken[b])] = page_of(i);
    }
    for (uint32_t i = first; i < n_give; i += stride) {
        const int b = owner(given, i), c = mapped(s, b);
        const int64_t top = static_cast<int64_t>(have0) + i;
        int page = s.table[static_cast<int64_t>(b) * s.max_pages + kept(s, b, c) + (i - given[b])];
        if (page < 0 || page >= s.num_pages) {   // no page: the entry keeps its place, which the sums have given it
            bad |= DSA_DEVERR_PAGE_RANGE;
            page = -1;
        }
        if (top < s.num_pages) s.free_pages[top] = page;
    }
    // ---- lengths and counts, a request a thread
    for (int b = blockIdx.x * kTabThreads + tid; b < s.B; b += gridDim.x * kTabThreads) {
        int len = 0, c = 0;
        if (__ldg(s.q_lens + b) >= 0) {
            const int64_t l = static_cast<int64_t>(max(0, __ldg(s.cached + b))) + (cu[b + 1] - cu[b]);
            len = static_cast<int>(min(l, static_cast<int64_t>(0x7fffffff)));
            const int got = max(0, min(static_cast<int>(taken[b + 1] - taken[b]), have - static_cast<int>(taken[b])));
            c = mapped(s, b) + got;
        }
        s.seq_lens[b] = len;
        s.counts_out[b] = c;
        s.cu_q[b] = static_cast<int32_t>(cu[b]);
    }
    if (blockIdx.x == 0 && tid == 0) {
        s.cu_q[s.B] = used;
        *s.free_count_out = have - static_cast<int>(min(n_take, static_cast<uint32_t>(have)));
    }
    if (bad != 0) raise_error(s.err, bad);
    ptx::griddep_launch_dependents();
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_step_tables(const int32_t* cached_lens, const int32_t* q_lens, const int32_t* page_counts,
                                      const int32_t* keep_pages, int32_t B, int32_t* block_table, int32_t max_pages,
                                      int64_t num_pages, int32_t* free_pages, const int32_t* free_count,
                                      int32_t* seq_lens, int32_t* page_counts_out, int32_t* free_count_out,
                                      int32_t* cu_q, int64_t* positions, int64_t* slot_mapping, int32_t T,
                                      int32_t* dev_err, void* stream) {
    using namespace dsa;
    if (B < 0 || T < 0 || max_pages < 0 || num_pages < 0) return DSA_ERR_INVALID_ARG;
    if (B == 0) return T == 0 ? DSA_OK : DSA_ERR_INVALID_ARG;
    if (max_pages < 1 || num_pages < 1) return DSA_ERR_INVALID_ARG;
    if (!cached_lens || !q_lens || !page_counts || !block_table || !free_pages || !free_count || !seq_lens ||
        !page_counts_out || !free_count_out || !cu_q)
        return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!positions || !slot_mapping)) return DSA_ERR_INVALID_ARG;
    if (B > kTabMaxRequests || num_pages * kPage >= 0x7fffffffLL || static_cast<int64_t>(B) * max_pages >= 0x7fffffffLL)
        return DSA_ERR_UNSUPPORTED;
    // every CTA reads all lengths at any time, and one writes what another reads nowhere: outputs lie apart
    const size_t nb = static_cast<size_t>(B) * 4, nt = static_cast<size_t>(T) * 8;
    struct Range { const void* p; size_t n; };
    const Range in[] = {{cached_lens, nb}, {q_lens, nb}, {page_counts, nb}, {keep_pages, nb}, {free_count, 4}};
    const Range out[] = {{block_table, nb * static_cast<size_t>(max_pages)}, {free_pages, static_cast<size_t>(num_pages) * 4},
                         {seq_lens, nb}, {page_counts_out, nb}, {free_count_out, 4}, {cu_q, nb + 4}, {positions, nt},
                         {slot_mapping, nt}};
    for (size_t i = 0; i < sizeof(out) / sizeof(out[0]); ++i) {
        for (const Range& r : in)
            if (overlap(out[i].p, out[i].n, r.p, r.n)) return DSA_ERR_INVALID_ARG;
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return DSA_ERR_INVALID_ARG;
    }
    const size_t smem = 3 * (static_cast<size_t>(B) + 1) * sizeof(uint32_t);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(3 * (kTabMaxRequests + 1) * sizeof(uint32_t))) != cudaSuccess)
        return DSA_ERR_CUDA;
    const int64_t want = std::max((static_cast<int64_t>(T) + kTabThreads - 1) / kTabThreads,
                                  (static_cast<int64_t>(B) + kTabWarps - 1) / kTabWarps);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), want))));
    cfg.blockDim = dim3(kTabThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const StepTables s{cached_lens, q_lens, page_counts, keep_pages, block_table, free_pages, free_count, seq_lens,
                       page_counts_out, free_count_out, cu_q, positions, slot_mapping, B, T, max_pages,
                       static_cast<int>(num_pages), dev_err};
    if (cudaLaunchKernelEx(&cfg, step_tables_kernel, s) != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}
