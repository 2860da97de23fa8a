// Writing rows of keys and values into the paged cache, quantising them on the
// way, and reading them back.
//
// Write.  A row is the D values of one token and head:
//   lo, hi = min, max;  s = fp16((hi - lo) / 2^bits);  z = fp16(lo);
//   c = clamp(floor((w - z) / s), 0, 2^bits - 1)
// (rtn.hpp).  D / 8 neighbouring lanes hold a row, 8 values each: one 16-byte
// load per lane of bf16 (two of fp32), the row's minimum and maximum from
// exchanges between the lanes, and one store of 8 codes per lane.  One pass
// over the data, nothing goes through LDS.
//
// Read.  The same lanes, the other way: 8 codes and the row's (s, z) in,
// s * (c + 1/2) + z out.  c + 1/2 has 9 bits and s 11, so the product is exact
// in fp32 and the fused sum rounds once.
//
// What bounds them.  Memory: 16381 tokens of 8 fp32 heads of 128 at 8 bits are
// written in 36 us (169 MB, 4.7 TB/s) and read back as bf16 in 19 us (101 MB, 5.4
// TB/s), with one division a row (kv_store.hpp).  A single token is a launch.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "kv_common.hpp"
#include "kv_store.hpp"

namespace grinqh {
namespace {

constexpr int kKvThreads = 256;
constexpr int kMaxKvGroups = 1 << 16;     // workgroups of a launch; more rows than they hold go round again

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct KvWriteArgs {
    KvDims d;
    const void* src[2];                   // keys, values
    uint8_t* codes[2];
    uint16_t* grid[2];
    const int64_t* slots;
    int64_t stride[2];                    // elements between tokens
    int n_tokens;
};

// Row r of one call's rows; the lanes of a row come here together.
template <int D, int BITS, typename T>
__device__ __forceinline__ void write_row(const KvWriteArgs& a, int which, int64_t r, int lane) {
    const int64_t token = r / a.d.heads;
    const int head = static_cast<int>(r - token * a.d.heads);
    const int64_t row = kv_row(a.d, a.slots[token], head);
    if (row < 0) return;
    const T* src = static_cast<const T*>(a.src[which]) + token * a.stride[which] + head * D + lane * kPerLane;
    float w[kPerLane];
    u32x4 raw = *reinterpret_cast<const u32x4*>(src);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = __uint_as_float(raw[i] << 16);
            w[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
        }
    } else {
        const u32x4 more = *reinterpret_cast<const u32x4*>(src + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __uint_as_float(raw[i]);
            w[4 + i] = __uint_as_float(more[i]);
        }
    }
    if constexpr (BITS == 16) {
        uint8_t* dst = a.codes[which] + row * (D * 2) + lane * (kPerLane * 2);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[i] = f32_to_bf16(w[2 * i]) | static_cast<uint32_t>(f32_to_bf16(w[2 * i + 1])) << 16;
        }
        *reinterpret_cast<u32x4*>(dst) = raw;
    } else {
        store_quantised_row<D, BITS>(w, a.codes[which], a.grid[which], row, lane);
    }
}

template <int D, int BITS, typename T>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(KvWriteArgs a) {
    constexpr int kLanes = D / kPerLane, kRows = kKvThreads / kLanes;
    const int64_t n_rows = static_cast<int64_t>(a.n_tokens) * a.d.heads;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kLanes; r < n_rows; r += step)
        write_row<D, BITS, T>(a, blockIdx.y, r, threadIdx.x % kLanes);
}

struct KvReadArgs {
    KvDims d;
    const uint8_t* codes[2];
    const uint16_t* grid[2];
    void* dst[2];
    const int64_t* slots;
    int n_tokens;
};

template <int D, int BITS, typename T>
__device__ __forceinline__ void read_row(const KvReadArgs& a, int which, int64_t r, int lane) {
    const int64_t token = r / a.d.heads;
    const int head = static_cast<int>(r - token * a.d.heads);
    const int64_t row = kv_row(a.d, a.slots[token], head);
    float w[kPerLane] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row >= 0) {
        const uint8_t* src = a.codes[which] + row * (D * BITS / 8) + lane * (kPerLane * BITS / 8);
        if constexpr (BITS == 16) {
            const u32x4 raw = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[2 * i] = __uint_as_float(raw[i] << 16);
                w[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
            }
        } else {
            uint32_t c[2];
            if constexpr (BITS == 8) {
                const u32x2 raw = *reinterpret_cast<const u32x2*>(src);
                c[0] = raw.x;
                c[1] = raw.y;
            } else {
                c[0] = *reinterpret_cast<const uint32_t*>(src);
            }
            const uint32_t g = *reinterpret_cast<const uint32_t*>(a.grid[which] + row * 2);
            const float s = f16_to_f32(static_cast<uint16_t>(g)), z = f16_to_f32(static_cast<uint16_t>(g >> 16));
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                const float q = static_cast<float>((c[i * BITS / 32] >> (i * BITS % 32)) & ((1u << BITS) - 1));
                w[i] = __builtin_fmaf(s, q + 0.5f, z);
            }
        }
    }
    T* dst = static_cast<T*>(a.dst[which]) + r * D + lane * kPerLane;
    u32x4 raw;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            raw[i] = f32_to_bf16(w[2 * i]) | static_cast<uint32_t>(f32_to_bf16(w[2 * i + 1])) << 16;
    } else {
        u32x4 more;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            raw[i] = __float_as_uint(w[i]);
            more[i] = __float_as_uint(w[4 + i]);
        }
        *reinterpret_cast<u32x4*>(dst + 4) = more;
    }
    *reinterpret_cast<u32x4*>(dst) = raw;
}

template <int D, int BITS, typename T>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvReadArgs a) {
    constexpr int kLanes = D / kPerLane, kRows = kKvThreads / kLanes;
    const int64_t n_rows = static_cast<int64_t>(a.n_tokens) * a.d.heads;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kLanes; r < n_rows; r += step)
        read_row<D, BITS, T>(a, blockIdx.y, r, threadIdx.x % kLanes);
}

bool aligned16(const void* p) { return aligned_to(p, 16); }

// Picks KERNEL<head_dim, bits, T> for a layout and value type.
template <template <int, int, typename> class Launch, typename Args>
grinqh_status dispatch(const grinqh_kv_layout& L, int dtype, dim3 grid, hipStream_t stream, const Args& a) {
    const auto by_bits = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        const auto by_type = [&](auto bits) {
            constexpr int B = decltype(bits)::value;
            return dtype == GRINQH_BF16 ? Launch<D, B, uint16_t>::run(grid, stream, a) : Launch<D, B, float>::run(grid, stream, a);
        };
        if (L.bits == 4) return by_type(std::integral_constant<int, 4>());
        if (L.bits == 8) return by_type(std::integral_constant<int, 8>());
        return by_type(std::integral_constant<int, 16>());
    };
    if (L.head_dim == 64) return by_bits(std::integral_constant<int, 64>());
    if (L.head_dim == 128) return by_bits(std::integral_constant<int, 128>());
    return by_bits(std::integral_constant<int, 256>());
}

template <int D, int B, typename T>
struct WriteLaunch {
    static grinqh_status run(dim3 grid, hipStream_t stream, const KvWriteArgs& a) {
        return launch_kernel(kv_write_kernel<D, B, T>, grid, kKvThreads, 0, stream, a);
    }
};

template <int D, int B, typename T>
struct ReadLaunch {
    static grinqh_status run(dim3 grid, hipStream_t stream, const KvReadArgs& a) {
        return launch_kernel(kv_read_kernel<D, B, T>, grid, kKvThreads, 0, stream, a);
    }
};

dim3 row_grid(const grinqh_kv_layout& L, int n_tokens) {
    const int64_t rows = static_cast<int64_t>(n_tokens) * L.n_kv_heads, per = kKvThreads * kPerLane / L.head_dim;
    return dim3(static_cast<unsigned>(std::min<int64_t>((rows + per - 1) / per, kMaxKvGroups)), 2);
}

}  // namespace

bool valid_kv_layout(const grinqh_kv_layout* L) {
    if (L == nullptr) return false;
    if (L->n_kv_heads < 1 || L->n_kv_heads > kMaxKvHeads) return false;
    if (L->head_dim != 64 && L->head_dim != 128 && L->head_dim != 256) return false;
    if (L->page_size != 16 && L->page_size != 32 && L->page_size != 64 && L->page_size != 128 && L->page_size != 256)
        return false;
    if (L->n_pages < 1 || L->n_pages > (1 << 24)) return false;
    if (L->bits != 4 && L->bits != 8 && L->bits != 16) return false;
    return L->row_bytes == L->head_dim * L->bits / 8;
}

grinqh_status check_kv_pools(const grinqh_kv_layout* L, const grinqh_kv_pools* p) {
    if (!valid_kv_layout(L) || p == nullptr || p->k_codes == nullptr || p->v_codes == nullptr) return GRINQH_EINVAL;
    if (L->bits < 16 && (p->k_grid == nullptr || p->v_grid == nullptr)) return GRINQH_EINVAL;
    if (!aligned16(p->k_codes) || !aligned16(p->v_codes)) return GRINQH_EALIGN;
    if (L->bits < 16 && (!aligned16(p->k_grid) || !aligned16(p->v_grid))) return GRINQH_EALIGN;
    return GRINQH_OK;
}

}  // namespace grinqh

using namespace grinqh;

extern "C" {

grinqh_status grinqh_kv_layout_init(int32_t n_kv_heads, int32_t head_dim, int32_t page_size, int32_t n_pages,
                                    int32_t bits, grinqh_kv_layout* out) {
    if (out == nullptr || bits < 0 || bits > 16 || head_dim < 0 || head_dim > 256) return GRINQH_EINVAL;
    const grinqh_kv_layout L{n_kv_heads, head_dim, page_size, n_pages, bits, head_dim * bits / 8};
    if (!valid_kv_layout(&L)) return GRINQH_EINVAL;
    *out = L;
    return GRINQH_OK;
}

size_t grinqh_kv_code_bytes(const grinqh_kv_layout* L) {
    if (!valid_kv_layout(L)) return 0;
    return static_cast<size_t>(L->n_pages) * L->n_kv_heads * L->page_size * L->row_bytes;
}

size_t grinqh_kv_grid_bytes(const grinqh_kv_layout* L) {
    if (!valid_kv_layout(L) || L->bits == 16) return 0;
    return static_cast<size_t>(L->n_pages) * L->n_kv_heads * L->page_size * 4u;
}

int64_t grinqh_debug_kv_row(const grinqh_kv_layout* L, int64_t slot, int32_t head) {
    if (!valid_kv_layout(L) || head < 0 || head >= L->n_kv_heads) return -1;
    return kv_row(kv_dims(*L), slot, head);
}

int64_t grinqh_debug_page_row(const grinqh_kv_layout* L, int32_t page, int32_t head, int32_t t) {
    if (!valid_kv_layout(L) || head < 0 || head >= L->n_kv_heads || t < 0) return -1;
    const KvDims d = kv_dims(*L);
    const int there = page_or_absent(page, d.n_pages);
    return there < 0 ? -1 - page_row(d, there, head, t) : page_row(d, there, head, t);
}

grinqh_status grinqh_kv_write(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const void* k,
                              const void* v, grinqh_dtype dtype, int64_t k_stride, int64_t v_stride,
                              int32_t n_tokens, const int64_t* slots, void* stream) {
    const grinqh_status st = check_kv_pools(L, pools);
    if (st != GRINQH_OK) return st;
    if ((dtype != GRINQH_BF16 && dtype != GRINQH_F32) || n_tokens < 0 || n_tokens > (1 << 24)) return GRINQH_EINVAL;
    if (n_tokens == 0) return GRINQH_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return GRINQH_EINVAL;
    const int64_t width = static_cast<int64_t>(L->n_kv_heads) * L->head_dim, eb = dtype == GRINQH_BF16 ? 2 : 4;
    if (k_stride < width || v_stride < width || k_stride > kMaxStride || v_stride > kMaxStride) return GRINQH_EINVAL;
    if (!aligned16(k) || !aligned16(v) || k_stride * eb % 16 != 0 || v_stride * eb % 16 != 0 ||
        reinterpret_cast<uintptr_t>(slots) % 8 != 0)
        return GRINQH_EALIGN;
    const size_t code_bytes = grinqh_kv_code_bytes(L), grid_bytes = grinqh_kv_grid_bytes(L);
    const auto rows = [&](int64_t stride) { return static_cast<size_t>(((n_tokens - 1) * stride + width) * eb); };
    if (written_overlaps({{pools->k_codes, code_bytes}, {pools->v_codes, code_bytes},      // keys and values at the same time
                          {pools->k_grid, grid_bytes}, {pools->v_grid, grid_bytes}},
                         {{k, rows(k_stride)}, {v, rows(v_stride)}, {slots, n_tokens * sizeof(int64_t)}}))
        return GRINQH_EINVAL;
    const KvWriteArgs a{kv_dims(*L), {k, v}, {pools->k_codes, pools->v_codes}, {pools->k_grid, pools->v_grid},
                        slots, {k_stride, v_stride}, n_tokens};
    return dispatch<WriteLaunch>(*L, dtype, row_grid(*L, n_tokens), static_cast<hipStream_t>(stream), a);
}

grinqh_status grinqh_kv_read(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const int64_t* slots,
                             int32_t n_tokens, void* k, void* v, grinqh_dtype dtype, void* stream) {
    const grinqh_status st = check_kv_pools(L, pools);
    if (st != GRINQH_OK) return st;
    if ((dtype != GRINQH_BF16 && dtype != GRINQH_F32) || n_tokens < 0 || n_tokens > (1 << 24)) return GRINQH_EINVAL;
    if (n_tokens == 0) return GRINQH_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return GRINQH_EINVAL;
    if (!aligned16(k) || !aligned16(v) || reinterpret_cast<uintptr_t>(slots) % 8 != 0) return GRINQH_EALIGN;
    const size_t n = static_cast<size_t>(n_tokens) * L->n_kv_heads * L->head_dim * (dtype == GRINQH_BF16 ? 2 : 4);
    const size_t code_bytes = grinqh_kv_code_bytes(L), grid_bytes = grinqh_kv_grid_bytes(L);
    if (written_overlaps({{k, n}, {v, n}}, {{slots, n_tokens * sizeof(int64_t)},
                                            {pools->k_codes, code_bytes}, {pools->v_codes, code_bytes},
                                            {pools->k_grid, grid_bytes}, {pools->v_grid, grid_bytes}}))
        return GRINQH_EINVAL;
    const KvReadArgs a{kv_dims(*L), {pools->k_codes, pools->v_codes}, {pools->k_grid, pools->v_grid}, {k, v},
                       slots, n_tokens};
    return dispatch<ReadLaunch>(*L, dtype, row_grid(*L, n_tokens), static_cast<hipStream_t>(stream), a);
}

}  // extern "C"
