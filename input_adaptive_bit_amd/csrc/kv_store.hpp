// Storing a row of the key-value cache from registers: D / 8 neighbouring lanes
// hold it, 8 values each.  Shared by the calls that write the cache.
#pragma once

#include "kv_common.hpp"
#include "rtn.hpp"

namespace grinqh {

constexpr int kPerLane = 8;               // values of a row per lane

// v of the lane that CTRL names, one for every lane.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// op over the D / 8 lanes of a row, the same bits in each of them.
template <int D, typename Op>
__device__ __forceinline__ float over_row(float v, Op op) {
    constexpr int kLanes = D / kPerLane;
    static_assert(kLanes == 8 || kLanes == 16 || kLanes == 32, "rows of 64, 128 or 256");
    v = op(v, dpp<0xB1>(v));                                  // lane ^ 1
    v = op(v, dpp<0x4E>(v));                                  // lane ^ 2
    v = op(v, dpp<0x141>(v));                                 // the other four of eight (mirrored)
    if constexpr (kLanes >= 16) v = op(v, dpp<0x140>(v));     // the other eight of sixteen (mirrored)
    if constexpr (kLanes == 32) v = op(v, __shfl_xor(v, 16, 32));
    return v;
}

// rtn_code for values that share s, with one division for all of them.  With
// r = 1 / s, u = d r is within 1.5 steps (of the 24-bit floats there) of d / s, and
// d - u s, 12 bits at most, is exact in a fused multiply-add; then u + (d - u s) r is
// 2^-23 steps off before it is rounded.  A border between two floats has 25 bits, s
// has 11 and d 24, so d / s is never on one and at least 2^-12 steps from it:
// the result is d / s rounded to nearest.  Only a quotient past 2^10 could overflow on
// the way, and d is cut down to that (the last code either way).  s = 0: r = 0, and
// so is the code.  An infinite s: NaN or 0, code 0 as well.
__device__ __forceinline__ uint32_t shared_scale_code(float w, float z, float s, float r, float top) {
    float d = w - z;
    d = d > 1024.f * s ? 1024.f * s : d;                      // a NaN stays one
    const float u = d * r;
    const float q = floorf(__builtin_fmaf(__builtin_fmaf(-u, s, d), r, u));
    return static_cast<uint32_t>(fminf(fmaxf(q, 0.f), top));  // a NaN becomes 0
}

// At 4 and 8 bits: the row's grid from its minimum and maximum (NaN ignored), then
// its codes.  The lanes of a row come here together.
template <int D, int BITS>
__device__ __forceinline__ void store_quantised_row(const float (&w)[kPerLane], uint8_t* codes, uint16_t* grid, int64_t row,
                                                    int lane) {
    typedef uint32_t two __attribute__((ext_vector_type(2)));
    uint8_t* dst = codes + row * (D * BITS / 8) + lane * (kPerLane * BITS / 8);
    float lo = w[0], hi = w[0];                               // fminf and fmaxf ignore NaN
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) {
        lo = fminf(lo, w[i]);
        hi = fmaxf(hi, w[i]);
    }
    lo = over_row<D>(lo, [](float x, float y) { return fminf(x, y); });
    hi = over_row<D>(hi, [](float x, float y) { return fmaxf(x, y); });
    const __half sh = rtn_scale(lo, hi, BITS), zh = rtn_zero(lo);
    const float s = __half2float(sh), z = __half2float(zh);
    constexpr float top = static_cast<float>((1 << BITS) - 1);
    const float r = s == 0.f ? 0.f : __fdiv_rn(1.f, s);
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const uint32_t q = shared_scale_code(w[i], z, s, r, top);
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
