// The key-value cache's addressing and row values, shared by the kernels that
// write, read and attend to it and by the host's checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

#include "device_common.hpp"
#include "grinqh.h"
#include "internal.h"

namespace grinqh {

// What a kernel needs of a layout (page_size is a power of two).
struct KvDims {
    int heads, page_shift, n_pages;
};

inline int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

inline KvDims kv_dims(const grinqh_kv_layout& L) { return KvDims{L.n_kv_heads, log2_of(L.page_size), L.n_pages}; }

// Row of (slot, head), or -1 for a slot outside the pool.  64 bits: a pool
// may hold more than 2^31 rows and 2^32 bytes.
__host__ __device__ __forceinline__ int64_t kv_row(const KvDims& d, int64_t slot, int head) {
    if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(d.n_pages) << d.page_shift) return -1;
    const int64_t page = slot >> d.page_shift;
    const int64_t t = slot & ((int64_t{1} << d.page_shift) - 1);
    return ((page * d.heads + head) << d.page_shift) + t;
}

// A page table's entry, or -1 where it names no page of the pool.
__host__ __device__ __forceinline__ int page_or_absent(int page, int n_pages) {
    return static_cast<unsigned>(page) < static_cast<unsigned>(n_pages) ? page : -1;
}

// Row of token t of a sequence in the page that holds it.  An absent page gives a
// row of page 0: the pool may be read there, and nothing of it is used.
__host__ __device__ __forceinline__ int64_t page_row(const KvDims& d, int page, int head, int t) {
    const int64_t at = page < 0 ? 0 : page;
    return ((at * d.heads + head) << d.page_shift) + (t & ((1 << d.page_shift) - 1));
}

// Largest sizes the calls accept.
constexpr int kMaxKvHeads = 1024, kMaxQHeads = 1024;
constexpr int64_t kMaxStride = int64_t{1} << 24;   // elements between tokens
constexpr int kMaxBatch = 1 << 20, kMaxCacheLen = 1 << 28, kMaxPacked = 1 << 24;

constexpr float kMaxScale = 1e30f;                 // times log2(e) it stays finite

// A launch that reports its own error and leaves none behind for the caller's
// next check (0.2 us sooner than <<<>>> and asking for the last error).
template <typename... P>
grinqh_status launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t lds, hipStream_t stream,
                            std::common_type_t<P>... args) {
    void* list[] = {&args...};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), list, lds, stream);
    if (e != hipSuccess) (void)hipGetLastError();
    return map_hip_error(e);
}

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && a0 < b0 + nb && b0 < a0 + na;
}

struct Span {
    const void* at;
    size_t bytes;
};

// Whether something that a call writes overlaps something that it reads or
// writes besides.
inline bool written_overlaps(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    for (const Span* w = written.begin(); w != written.end(); ++w) {
        for (const Span& r : read)
            if (overlaps(w->at, w->bytes, r.at, r.bytes)) return true;
        for (const Span* x = w + 1; x != written.end(); ++x)
            if (overlaps(w->at, w->bytes, x->at, x->bytes)) return true;
    }
    return false;
}

bool valid_kv_layout(const grinqh_kv_layout* L);
// Host checks of a cache: GRINQH_OK, or the status a call returns.
grinqh_status check_kv_pools(const grinqh_kv_layout* L, const grinqh_kv_pools* pools);

__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));   // round to nearest even
}

}  // namespace grinqh
