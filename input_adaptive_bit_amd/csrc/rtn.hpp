// Round-to-nearest onto the midpoint grid s * (q + 1/2) + z (key design 3 at
// full width): the rounding rules shared by the weight quantiser
// (quantize.hip) and the key-value cache (kv_cache.hip).
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace grinqh {

// s = fp16((hi - lo) / 2^bits), a zero as +0.
__device__ __forceinline__ __half rtn_scale(float lo, float hi, int bits) {
    return __float2half_rn((hi - lo) * __uint_as_float(static_cast<uint32_t>(127 - bits) << 23) + 0.f);
}

// z = fp16(lo), a zero as +0.
__device__ __forceinline__ __half rtn_zero(float lo) { return __float2half_rn(lo + 0.f); }

// min(max(floor((w - z) / s), 0), top) with an IEEE division; a NaN quotient
// gives 0.  The caller gives 0 itself where s = 0.
__device__ __forceinline__ uint8_t rtn_code(float w, float z, float s, float top) {
    float u = floorf(__fdiv_rn(w - z, s));
    u = fmaxf(u, 0.f);                         // a NaN quotient becomes 0 here
    u = fminf(u, top);
    return static_cast<uint8_t>(u);
}

}  // namespace grinqh
