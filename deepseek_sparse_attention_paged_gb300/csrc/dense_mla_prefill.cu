// dense_mla_prefill.cu -- attention of a prompt in expanded form: per-head keys and values made from
// the latent rows, one rope key shared by all heads.
//
// Follows vllm mla/common.py, MLACommonImpl._forward_prefill (k = [k_nope, k_pe], causal attention
// over ragged requests) and _compute_prefill_context (a chunk's queries over earlier keys).
//
// S_ij = scale (<q_i[0:128], k_nope_j> + <q_i[128:192], k_pe_j>), O = softmax(S) V.  One warp per
// (row, head); running maximum and sum, fp32 accumulation.
#include <cuda_bf16.h>

#include "dsa_common.cuh"

namespace dsa {
namespace {

constexpr int kPreThreads = 256;

struct Strided {
    const uint16_t* p;
    int64_t row, head;
};

__device__ __forceinline__ float2 pair_at(const uint16_t* p, int lane) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p) + lane);
    return make_float2(bf16_lo(w), bf16_hi(w));
}

__global__ void __launch_bounds__(kPreThreads)
dense_mla_prefill_kernel(Strided q, Strided k, Strided pe, Strided val, const int32_t* __restrict__ cu_q,
                         const int32_t* __restrict__ cu_k, int B, int T, int S, int H, float scale, int causal,
                         uint16_t* __restrict__ out, int64_t out_row, int64_t out_head, float* __restrict__ lse,
                         int32_t* err) {
    const int64_t rh = (static_cast<int64_t>(blockIdx.x) * kPreThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int r = static_cast<int>(rh / H), h = static_cast<int>(rh % H);
    if (r >= T || r >= __ldg(cu_q + B)) return;
    const int b = row_request(cu_q, B, r);
    const int q0 = __ldg(cu_q + b), k0 = max(0, __ldg(cu_k + b)), k1 = __ldg(cu_k + b + 1);
    const int q1 = __ldg(cu_q + b + 1);
    const int nq = min(q1, T) - q0;
    if (q1 > T && lane == 0) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    if (k0 < 0 || k1 < k0 || k1 > S) {
        if (lane == 0) raise_error(err, DSA_DEVERR_INDEX_RANGE);
    }
    const int nk = max(0, min(k1, S) - k0);   // keys k0 .. k0 + nk - 1
    const int vis = causal ? max(0, nk - nq + (r - q0) + 1) : nk;
    float2 qv[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        qv[c] = pair_at(q.p + r * q.row + h * q.head + c * 64, lane);
        qv[c].x *= scale;
        qv[c].y *= scale;
    }
    float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < vis; ++j) {
        const int64_t row = k0 + j;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            const float2 kk = pair_at(c < 2 ? k.p + row * k.row + h * k.head + c * 64 : pe.p + row * pe.row, lane);
            s = fmaf(qv[c].x, kk.x, fmaf(qv[c].y, kk.y, s));
        }
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float a = expf(m - mn), e = expf(s - mn);
        l = l * a + e;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float2 vv = pair_at(val.p + row * val.row + h * val.head + c * 64, lane);
            acc[2 * c] = acc[2 * c] * a + e * vv.x;
            acc[2 * c + 1] = acc[2 * c + 1] * a + e * vv.y;
        }
        m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const __nv_bfloat162 o = __floats2bfloat162_rn(acc[2 * c] * inv, acc[2 * c + 1] * inv);
        reinterpret_cast<uint32_t*>(out + r * out_row + h * out_head + c * 64)[lane] =
            *reinterpret_cast<const uint32_t*>(&o);
    }
    if (lse != nullptr && lane == 0) lse[rh] = l > 0.0f ? m + logf(l) : -INFINITY;
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
    if (static_cast<int64_t>(T) * H >= 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
    const int64_t warps = static_cast<int64_t>(T) * H;
    dense_mla_prefill_kernel<<<static_cast<unsigned>((warps * 32 + kPreThreads - 1) / kPreThreads), kPreThreads, 0,
                               static_cast<cudaStream_t>(stream)>>>(
        Strided{static_cast<const uint16_t*>(q_bf16), q_row_stride, q_head_stride},
        Strided{static_cast<const uint16_t*>(k_nope_bf16), k_row_stride, k_head_stride},
        Strided{static_cast<const uint16_t*>(k_pe_bf16), pe_row_stride, 0},
        Strided{static_cast<const uint16_t*>(v_bf16), v_row_stride, v_head_stride}, cu_q, cu_k, B, T, S, H, scale,
        (flags & DSA_CAUSAL) ? 1 : 0, static_cast<uint16_t*>(out_bf16), out_row_stride, out_head_stride, lse, dev_err);
    return launch_status();
}
