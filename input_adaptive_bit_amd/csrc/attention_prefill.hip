// Attention over whole prompts, packed behind one another, with grouped heads.
//
// For query i of a sequence with n queries and m keys, and key-value head
// g = h / group,
//   o = sum_j p_j v_j,  p_j = exp(a_j - max) / sum,  a_j = scale * q . k_j,
// over the keys j <= i + m - n (all keys where not causal).
//
// One wave per (query, head) walks the keys 64 at a time with the running
// maximum and sum.
#include <math.h>

#include "internal.h"
#include "kv_common.hpp"

namespace grinqh {
namespace {

typedef grinqh_prefill_attention_args Args;

template <int D>
__global__ __launch_bounds__(kWave) void prefill_attention_kernel(Args a) {
    constexpr int kOwn = D / kWave;
    const int row = blockIdx.x, h = blockIdx.y, g = h / (a.n_q_heads / a.n_kv_heads), lane = threadIdx.x;
    int b = 0, q_begin = 0, q_end = 0;
    for (; b < a.batch; ++b) {                        // the sequence that holds the row
        q_begin = min(max(a.cu_q[b], 0), a.total_q);
        q_end = min(max(a.cu_q[b + 1], 0), a.total_q);
        if (row >= q_begin && row < q_end) break;
    }
    if (b == a.batch) return;
    const int k_begin = min(max(a.cu_k[b], 0), a.total_k), k_end = min(max(a.cu_k[b + 1], 0), a.total_k);
    const int n = q_end - q_begin, keys = max(k_end - k_begin, 0), i = row - q_begin;
    const int seen = a.causal ? max(min(i + keys - n + 1, keys), 0) : keys;
    __shared__ float qs[D], ps[kWave];
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + row * a.q_stride + h * D;
    const uint16_t* k = static_cast<const uint16_t*>(a.k) + k_begin * a.k_stride + g * D;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + k_begin * a.v_stride + g * D;
    for (int d = lane; d < D; d += kWave) qs[d] = bf16_to_f32(q[d]);
    float m = -INFINITY, l = 0.f, o[kOwn];
    for (int x = 0; x < kOwn; ++x) o[x] = 0.f;
    for (int t0 = 0; t0 < seen; t0 += kWave) {
        const int t = t0 + lane;
        __syncthreads();
        float score = -INFINITY;
        if (t < seen) {
            float sum = 0.f;
            for (int d = 0; d < D; ++d) sum = __builtin_fmaf(qs[d], bf16_to_f32(k[t * a.k_stride + d]), sum);
            score = sum * a.scale;
        }
        float top = score;
        for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.f : m_new;
        const float p = t < seen ? expf(score - base) : 0.f, keep = expf(m - base);
        float total = p;
        for (int x = 1; x < kWave; x <<= 1) total += __shfl_xor(total, x);
        l = l * keep + total;
        m = m_new;
        ps[lane] = p;
        __syncthreads();
        for (int x = 0; x < kOwn; ++x) o[x] *= keep;
        for (int j = 0; j < min(kWave, seen - t0); ++j)
            for (int x = 0; x < kOwn; ++x)
                o[x] = __builtin_fmaf(ps[j], bf16_to_f32(v[(t0 + j) * a.v_stride + lane + x * kWave]), o[x]);
    }
    const int64_t o0 = (static_cast<int64_t>(row) * a.n_q_heads + h) * D;
    for (int x = 0; x < kOwn; ++x) {
        const float y = l == 0.f ? 0.f : o[x] / l;
        if (a.out_dtype == GRINQH_F32)
            static_cast<float*>(a.out)[o0 + lane + x * kWave] = y;
        else
            static_cast<uint16_t*>(a.out)[o0 + lane + x * kWave] = f32_to_bf16(y);
    }
    if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(row) * a.n_q_heads + h] = m + logf(l);
}

}  // namespace
}  // namespace grinqh

using namespace grinqh;

extern "C" grinqh_status grinqh_prefill_attention(const grinqh_prefill_attention_args* args, void* stream) {
    if (args == nullptr) return GRINQH_EINVAL;
    const Args& a = *args;
    if (a.batch < 0 || a.batch > kMaxBatch || a.total_q < 0 || a.total_q > kMaxPacked || a.total_k < 0 ||
        a.total_k > kMaxPacked)
        return GRINQH_EINVAL;
    if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return GRINQH_EINVAL;
    if (a.n_kv_heads < 1 || a.n_kv_heads > kMaxKvHeads || a.n_q_heads < 1 || a.n_q_heads > kMaxQHeads ||
        a.n_q_heads % a.n_kv_heads != 0 || !isfinite(a.scale))
        return GRINQH_EINVAL;
    if (a.out_dtype != GRINQH_BF16 && a.out_dtype != GRINQH_F32) return GRINQH_EINVAL;
    if (a.batch == 0 || a.total_q == 0) return GRINQH_OK;
    if (a.q == nullptr || a.cu_q == nullptr || a.cu_k == nullptr || a.out == nullptr) return GRINQH_EINVAL;
    if (a.total_k > 0 && (a.k == nullptr || a.v == nullptr)) return GRINQH_EINVAL;
    const int64_t qw = static_cast<int64_t>(a.n_q_heads) * a.head_dim, kw = static_cast<int64_t>(a.n_kv_heads) * a.head_dim;
    if (a.q_stride < qw || a.k_stride < kw || a.v_stride < kw || a.q_stride > kMaxStride || a.k_stride > kMaxStride ||
        a.v_stride > kMaxStride)
        return GRINQH_EINVAL;
    if (!aligned_to(a.q, 16) || !aligned_to(a.k, 16) || !aligned_to(a.v, 16) || a.q_stride % 8 != 0 ||
        a.k_stride % 8 != 0 || a.v_stride % 8 != 0 || !aligned_to(a.cu_q, 4) || !aligned_to(a.cu_k, 4) ||
        !aligned_to(a.out, 16) || !aligned_to(a.lse, 4))
        return GRINQH_EALIGN;
    const size_t out_bytes = static_cast<size_t>(a.total_q) * qw * (a.out_dtype == GRINQH_BF16 ? 2 : 4);
    if (overlaps(a.q, static_cast<size_t>((a.total_q - 1) * a.q_stride + qw) * 2, a.out, out_bytes)) return GRINQH_EINVAL;
    if (a.total_k > 0 &&
        (overlaps(a.k, static_cast<size_t>((a.total_k - 1) * a.k_stride + kw) * 2, a.out, out_bytes) ||
         overlaps(a.v, static_cast<size_t>((a.total_k - 1) * a.v_stride + kw) * 2, a.out, out_bytes)))
        return GRINQH_EINVAL;
    DeviceInfo dev;
    hipError_t e;
    if (!current_device_info(&dev, &e)) return map_hip_error(e);
    const dim3 grid(static_cast<unsigned>(a.total_q), static_cast<unsigned>(a.n_q_heads));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.head_dim == 64) prefill_attention_kernel<64><<<grid, dim3(kWave), 0, s>>>(a);
    else if (a.head_dim == 128) prefill_attention_kernel<128><<<grid, dim3(kWave), 0, s>>>(a);
    else prefill_attention_kernel<256><<<grid, dim3(kWave), 0, s>>>(a);
    return map_hip_error(hipGetLastError());
}
