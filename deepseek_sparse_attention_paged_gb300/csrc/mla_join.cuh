// mla_join.cuh -- joins the parts of split row tiles of the dense latent attention behind shared prefixes: fp32 results over
// disjoint key ranges, each normalised, with their log-sum-exp (base 2).
#pragma once

#include "attn_common.cuh"

namespace dsa {
namespace attn {

constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 4;     // per SM

// A split row tile: its first output row and number of rows (0: none), and its parts: the first in the row of slots
// `slot` + 1, the j-th in `slot` + j `step`.
struct JoinTask {
    int64_t out_row;
    int rows, parts, slot, step;
};

// V x 128 dims from d0 on of one output row, joined from n parts, P at a time: their sums and values are loaded
// together.  slot_of(j): the row of part j.
template <int V, int P, typename F>
__device__ __forceinline__ void join_row(const float* __restrict__ part_o, const float* __restrict__ part_lse, int n,
                                         F slot_of, int64_t out_row, int d0, int lane, uint16_t* __restrict__ out,
                                         float* __restrict__ lse_out) {
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
        *reinterpret_cast<uint2*>(out + out_row * kValueDim + d0 + v * 128 + lane * 4) =
            make_uint2(pack_bf16x2(acc[v].x * inv, acc[v].y * inv), pack_bf16x2(acc[v].z * inv, acc[v].w * inv));
    if (lse_out != nullptr && d0 == 0 && lane == 0)
        lse_out[out_row] = tot == 0.0f ? -INFINITY : (m_run + log2f(tot)) * kLn2;
}

// All split row tiles, task(c) for c < candidates.  Bound by the latency of its loads: 128 dims of an output row a warp, four
// parts at a time, when there are few rows, and a whole row, two parts at a time, when there are many.
template <typename F>
__device__ __forceinline__ void join_listed(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                            int candidates, int slot_rows, uint16_t* __restrict__ out,
                                            float* __restrict__ lse_out, F task) {
    // the row tiles to join, read at once (one after the other they would cost a memory latency each) and
    // listed in order, so that every block counts alike
    __shared__ JoinTask list[kJoinThreads];
    __shared__ int found[kJoinThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nwarps = gridDim.x * (kJoinThreads / 32);
    const int first = blockIdx.x * (kJoinThreads / 32) + warp;
    for (int c0 = 0; c0 < candidates; c0 += kJoinThreads) {
        JoinTask own{0, 0, 0, 0, 0};
        if (c0 + static_cast<int>(threadIdx.x) < candidates) own = task(c0 + static_cast<int>(threadIdx.x));
        const uint32_t mask = __ballot_sync(0xffffffffu, own.rows > 0);
        if (lane == 0) found[warp] = __popc(mask);
        __syncthreads();
        int total = 0, before = 0;
        for (int i = 0; i < kJoinThreads / 32; ++i) {
            if (i == warp) before = total;
            total += found[i];
        }
        if (own.rows > 0) {
            const int j = before + __popc(mask & ((1u << lane) - 1u));
            list[j] = own;
        }
        __syncthreads();
        const bool many = 2 * total * slot_rows >= nwarps;
        int at = first;                                                   // this warp's next task, counted over the list
        for (int li = 0; li < total; ++li) {
            const JoinTask m = list[li];
            const int tasks = many ? m.rows : m.rows * 4;
            for (; at < tasks; at += nwarps) {
                const int row = many ? at : at >> 2;
                auto slot_of = [&](int j) {
                    return static_cast<int64_t>(j == 0 ? m.slot + 1 : m.slot + j * m.step) * slot_rows + row;
                };
                if (many) join_row<4, 2>(part_o, part_lse, m.parts, slot_of, m.out_row + row, 0, lane, out, lse_out);
                else join_row<1, 4>(part_o, part_lse, m.parts, slot_of, m.out_row + row, (at & 3) * 128, lane, out, lse_out);
            }
            at -= tasks;
        }
        __syncthreads();
    }
}

}  // namespace attn
}  // namespace dsa
