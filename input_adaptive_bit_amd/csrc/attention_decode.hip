// Attention of one new token of every sequence over its paged key-value cache.
//
// For query head h with key-value head g = h / group,
//   o = sum_t p_t v_t,  p_t = exp(a_t - m) / l,  a_t = scale * q . k_t.
//
// One wave per (sequence, query head) walks the tokens 64 at a time with the
// running maximum m and sum l: a lane forms one token's score, then every
// lane owns D / 64 values of the output and adds the 64 tokens' values to them.
#include <math.h>

#include "internal.h"
#include "kv_common.hpp"

namespace grinqh {
namespace {

struct DecodeArgs {
    KvDims d;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint16_t* k_grid;
    const uint16_t* v_grid;
    const void* q;
    const int32_t* page_table;
    const int32_t* seq_lens;
    void* out;
    float* lse;
    int64_t q_stride, table_stride;
    int n_q_heads, group, longest, q_dtype, out_dtype;   // longest: min(max_len, max_pages * page_size)
    float scale;
};

template <int BITS>
__device__ __forceinline__ float cached(const uint8_t* codes, float s, float z, int d) {
    if constexpr (BITS == 16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(codes)[d]);
    const int c = BITS == 8 ? codes[d] : (codes[d >> 1] >> (4 * (d & 1))) & 15;
    return __builtin_fmaf(s, static_cast<float>(c) + 0.5f, z);
}

template <int D, int BITS>
__global__ __launch_bounds__(kWave) void decode_kernel(DecodeArgs a) {
    constexpr int kRow = D * BITS / 8, kOwn = D / kWave;
    const int64_t item = blockIdx.x;
    const int b = static_cast<int>(item / a.n_q_heads), h = static_cast<int>(item % a.n_q_heads), g = h / a.group;
    const int lane = threadIdx.x;
    __shared__ float qs[D], ps[kWave];
    __shared__ int64_t rows[kWave];
    const int64_t q0 = b * a.q_stride + static_cast<int64_t>(h) * D;
    for (int d = lane; d < D; d += kWave)
        qs[d] = a.q_dtype == GRINQH_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(a.q)[q0 + d])
                                         : static_cast<const float*>(a.q)[q0 + d];
    __syncthreads();
    const int len = min(max(a.seq_lens[b], 0), a.longest);
    float m = -INFINITY, l = 0.f, o[kOwn];
    for (int i = 0; i < kOwn; ++i) o[i] = 0.f;
    for (int t0 = 0; t0 < len; t0 += kWave) {
        const int t = t0 + lane;
        int64_t row = -1;
        if (t < len) {
            const int64_t page = a.page_table[b * a.table_stride + (t >> a.d.page_shift)];
            row = kv_row(a.d, (page << a.d.page_shift) + (t & ((1 << a.d.page_shift) - 1)), g);
        }
        float score = -INFINITY;
        if (row >= 0) {
            float s = 0.f, z = 0.f, sum = 0.f;
            if (BITS < 16) {
                s = f16_to_f32(a.k_grid[2 * row]);
                z = f16_to_f32(a.k_grid[2 * row + 1]);
            }
            for (int d = 0; d < D; ++d) sum = __builtin_fmaf(qs[d], cached<BITS>(a.k_codes + row * kRow, s, z, d), sum);
            score = sum * a.scale;
        }
        float top = score;
        for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.f : m_new;
        const float p = row >= 0 ? expf(score - base) : 0.f, keep = expf(m - base);
        float total = p;
        for (int x = 1; x < kWave; x <<= 1) total += __shfl_xor(total, x);
        l = l * keep + total;
        m = m_new;
        __syncthreads();
        ps[lane] = p;
        rows[lane] = row;
        __syncthreads();
        for (int i = 0; i < kOwn; ++i) o[i] *= keep;
        for (int j = 0; j < min(kWave, len - t0); ++j) {
            const int64_t r = rows[j];
            if (r < 0) continue;
            float s = 0.f, z = 0.f;
            if (BITS < 16) {
                s = f16_to_f32(a.v_grid[2 * r]);
                z = f16_to_f32(a.v_grid[2 * r + 1]);
            }
            for (int i = 0; i < kOwn; ++i)
                o[i] = __builtin_fmaf(ps[j], cached<BITS>(a.v_codes + r * kRow, s, z, lane + i * kWave), o[i]);
        }
    }
    const int64_t o0 = (static_cast<int64_t>(b) * a.n_q_heads + h) * D;
    for (int i = 0; i < kOwn; ++i) {
        const float y = l == 0.f ? 0.f : o[i] / l;
        if (a.out_dtype == GRINQH_F32)
            static_cast<float*>(a.out)[o0 + lane + i * kWave] = y;
        else
            static_cast<uint16_t*>(a.out)[o0 + lane + i * kWave] = f32_to_bf16(y);
    }
    if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(b) * a.n_q_heads + h] = m + logf(l);
}

template <int D>
void launch_bits(const DecodeArgs& a, int bits, unsigned n, hipStream_t stream) {
    if (bits == 4) decode_kernel<D, 4><<<dim3(n), dim3(kWave), 0, stream>>>(a);
    else if (bits == 8) decode_kernel<D, 8><<<dim3(n), dim3(kWave), 0, stream>>>(a);
    else decode_kernel<D, 16><<<dim3(n), dim3(kWave), 0, stream>>>(a);
}

bool valid_heads(const grinqh_kv_layout* L, int n_q_heads, int batch, int max_len) {
    return valid_kv_layout(L) && n_q_heads >= 1 && n_q_heads <= kMaxQHeads && n_q_heads % L->n_kv_heads == 0 &&
           batch >= 0 && batch <= kMaxBatch && max_len >= 1 && max_len <= kMaxCacheLen;
}

}  // namespace
}  // namespace grinqh

using namespace grinqh;

extern "C" {

size_t grinqh_attention_workspace_bytes(const grinqh_kv_layout* L, int32_t n_q_heads, int32_t batch,
                                        int32_t max_len) {
    if (!valid_heads(L, n_q_heads, batch, max_len)) return 0;
    return 256;
}

grinqh_status grinqh_decode_attention(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const void* q,
                                      grinqh_dtype q_dtype, int64_t q_stride, int32_t n_q_heads,
                                      const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                      const int32_t* seq_lens, int32_t batch, int32_t max_len, float scale,
                                      void* out, grinqh_dtype out_dtype, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    const grinqh_status st = check_kv_pools(L, pools);
    if (st != GRINQH_OK) return st;
    if (!valid_heads(L, n_q_heads, batch, max_len) || !isfinite(scale)) return GRINQH_EINVAL;
    if ((q_dtype != GRINQH_BF16 && q_dtype != GRINQH_F32) || (out_dtype != GRINQH_BF16 && out_dtype != GRINQH_F32))
        return GRINQH_EINVAL;
    if (batch == 0) return GRINQH_OK;
    if (q == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr || workspace == nullptr)
        return GRINQH_EINVAL;
    const int64_t width = static_cast<int64_t>(n_q_heads) * L->head_dim;
    if (q_stride < width || q_stride > kMaxStride || max_pages < 1 || table_stride < max_pages ||
        table_stride > kMaxStride)
        return GRINQH_EINVAL;
    const int64_t qb = q_dtype == GRINQH_BF16 ? 2 : 4, ob = out_dtype == GRINQH_BF16 ? 2 : 4;
    if (!aligned_to(q, 16) || q_stride * qb % 16 != 0 || !aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) ||
        !aligned_to(out, 16) || !aligned_to(lse, 4) || !aligned_to(workspace, 256))
        return GRINQH_EALIGN;
    if (workspace_bytes < grinqh_attention_workspace_bytes(L, n_q_heads, batch, max_len)) return GRINQH_ENOSPACE;
    if (overlaps(q, static_cast<size_t>(((batch - 1) * q_stride + width) * qb), out,
                 static_cast<size_t>(batch * width * ob)))
        return GRINQH_EINVAL;
    DeviceInfo dev;
    hipError_t e;
    if (!current_device_info(&dev, &e)) return map_hip_error(e);
    const int64_t reach = static_cast<int64_t>(max_pages) * L->page_size;
    const DecodeArgs a{kv_dims(*L), pools->k_codes, pools->v_codes, pools->k_grid, pools->v_grid, q, page_table,
                       seq_lens, out, lse, q_stride, table_stride, n_q_heads, n_q_heads / L->n_kv_heads,
                       static_cast<int>(reach < max_len ? reach : max_len), q_dtype, out_dtype, scale};
    const unsigned n = static_cast<unsigned>(batch) * n_q_heads;
    if (L->head_dim == 64) launch_bits<64>(a, L->bits, n, static_cast<hipStream_t>(stream));
    else if (L->head_dim == 128) launch_bits<128>(a, L->bits, n, static_cast<hipStream_t>(stream));
    else launch_bits<256>(a, L->bits, n, static_cast<hipStream_t>(stream));
    return map_hip_error(hipGetLastError());
}

}  // extern "C"
