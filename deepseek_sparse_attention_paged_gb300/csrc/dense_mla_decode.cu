// dense_mla_decode.cu -- absorbed latent attention of new tokens over the whole paged latent cache.
//
// Follows vllm mla/common.py, MLACommonImpl.forward decode branch (_forward_decode on the absorbed
// query [ql_nope 512, q_pe 64] and the paged latent cache; returns (out, lse)).
//
// S_j = scale <q[r,h], C[j]> over the v_r visible positions, out = softmax(S) C[:, 0:512].
// One warp per (row, head): lane l holds dims 2 l, 2 l + 1 of each of the 9 64-dim chunks; running
// maximum and sum, fp32 accumulation.
#include <cuda_bf16.h>

#include "dsa_common.cuh"

namespace dsa {
namespace {

constexpr int kDecThreads = 256;

__global__ void __launch_bounds__(kDecThreads)
dense_mla_decode_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ kv, int64_t num_pages,
                        const int32_t* __restrict__ block_table, int max_pages, const int32_t* __restrict__ seq_lens,
                        const int32_t* __restrict__ cu_q, int B, int T, int H, float scale,
                        uint16_t* __restrict__ out, float* __restrict__ lse, int32_t* err) {
    const int64_t rh = (static_cast<int64_t>(blockIdx.x) * kDecThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int r = static_cast<int>(rh / H);
    if (r >= T || r >= __ldg(cu_q + B)) return;
    const int b = row_request(cu_q, B, r);
    const int q0 = __ldg(cu_q + b);
    const int q1 = __ldg(cu_q + b + 1);
    if (q1 > T && lane == 0) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    int v = visible_len(__ldg(seq_lens + b), min(q1, T) - q0, r - q0);
    if (v > max_pages * kPage) {
        v = max_pages * kPage;
        if (lane == 0) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    }
    float qv[18], acc[16];
#pragma unroll
    for (int c = 0; c < 9; ++c) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q + rh * kLatentDim + c * 64) + lane);
        qv[2 * c] = bf16_lo(w) * scale;
        qv[2 * c + 1] = bf16_hi(w) * scale;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int p = 0; p < v; ++p) {
        const int page = __ldg(block_table + static_cast<int64_t>(b) * max_pages + (p >> 6));
        if (page < 0 || page >= num_pages) {
            if (lane == 0) raise_error(err, DSA_DEVERR_PAGE_RANGE);
            continue;
        }
        const uint16_t* row = kv + (static_cast<int64_t>(page) * kPage + (p & 63)) * kLatentDim;
        float k[18], s = 0.0f;
#pragma unroll
        for (int c = 0; c < 9; ++c) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row + c * 64) + lane);
            k[2 * c] = bf16_lo(w);
            k[2 * c + 1] = bf16_hi(w);
            s = fmaf(qv[2 * c], k[2 * c], fmaf(qv[2 * c + 1], k[2 * c + 1], s));
        }
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float a = expf(m - mn), e = expf(s - mn);
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = acc[i] * a + e * k[i];
        m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const __nv_bfloat162 o = __floats2bfloat162_rn(acc[2 * c] * inv, acc[2 * c + 1] * inv);
        reinterpret_cast<uint32_t*>(out + rh * kValueDim + c * 64)[lane] = *reinterpret_cast<const uint32_t*>(&o);
    }
    if (lse != nullptr && lane == 0) lse[rh] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace dsa

extern "C" size_t dsa_dense_mla_decode_workspace_size(int32_t T, int32_t H) {
    (void)T;
    (void)H;
    return 0;
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
    if (num_pages * kPage >= 0x7fffffffLL || static_cast<int64_t>(max_pages) * kPage >= 0x7fffffffLL ||
        static_cast<int64_t>(T) * H >= 0x7fffffffLL)
        return DSA_ERR_UNSUPPORTED;
    const size_t need = dsa_dense_mla_decode_workspace_size(T, H);
    if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need)) return DSA_ERR_INVALID_ARG;
    const int64_t warps = static_cast<int64_t>(T) * H;
    dense_mla_decode_kernel<<<static_cast<unsigned>((warps * 32 + kDecThreads - 1) / kDecThreads), kDecThreads, 0,
                              static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t*>(q_bf16), static_cast<const uint16_t*>(kv_pool), num_pages, block_table, max_pages,
        seq_lens, cu_q, B, T, H, scale, static_cast<uint16_t*>(out_bf16), lse, dev_err);
    return launch_status();
}
