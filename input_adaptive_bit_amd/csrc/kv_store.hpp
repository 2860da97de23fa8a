// Storing a row of the key-value cache from registers: D / 8 neighbouring lanes
// hold it, 8 values each.  Shared by the calls that write the cache.
#pragma once

#include "kv_common.hpp"
#include "rtn.hpp"

namespace grinqh {

constexpr int kPerLane = 8;               // values of a row per lane

// At 4 and 8 bits: the row's grid from its minimum and maximum (NaN ignored), then
// its codes.  The lanes of a row come here together.
template <int D, int BITS>
__device__ __forceinline__ void store_quantised_row(const float (&w)[kPerLane], uint8_t* codes, uint16_t* grid, int64_t row,
                                                    int lane) {
    typedef uint32_t two __attribute__((ext_vector_type(2)));
    constexpr int kLanes = D / kPerLane;
    uint8_t* dst = codes + row * (D * BITS / 8) + lane * (kPerLane * BITS / 8);
    float lo = w[0], hi = w[0];                               // fminf and fmaxf ignore NaN
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) {
        lo = fminf(lo, w[i]);
        hi = fmaxf(hi, w[i]);
    }
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, m, kLanes));
        hi = fmaxf(hi, __shfl_xor(hi, m, kLanes));
    }
    const __half sh = rtn_scale(lo, hi, BITS), zh = rtn_zero(lo);
    const float s = __half2float(sh), z = __half2float(zh);
    constexpr float top = static_cast<float>((1 << BITS) - 1);
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const uint32_t q = s == 0.f ? 0u : rtn_code(w[i], z, s, top);
        c[i * BITS / 32] |= q << (i * BITS % 32);
    }
    if constexpr (BITS == 8)
        *reinterpret_cast<two*>(dst) = two{c[0], c[1]};
    else
        *reinterpret_cast<uint32_t*>(dst) = c[0];
    if (lane == 0)
        *reinterpret_cast<uint32_t*>(grid + row * 2) =
            __half_as_ushort(sh) | static_cast<uint32_t>(__half_as_ushort(zh)) << 16;
}

}  // namespace grinqh
