// fa_e4m3.cuh -- 8-bit cache rows: e4m3 values times a power of two per row (device helpers).
//
// A row x of D values is held as q_i = e4m3(x_i * 2^-e) and the byte e + 127, where e is the
// smallest integer with max|x| <= 448 * 2^e (448 is e4m3's largest value), clamped to
// [-127, 127].  A power of two costs a floating-point format nothing in relative precision and
// makes the scaling exact, so each value is rounded once (to nearest, ties to even) and
// reading back is exact in bf16 and, inside its range, in fp16.  A row that holds an infinity or
// a NaN has no such e: its byte is 255 and it reads back as NaN.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace fa {

constexpr uint32_t kExpNan = 255;

// Biased exponent of a row from the largest of its values' fp32 bit patterns without the sign
// (ordered like the magnitudes, with NaN above infinity).  448 = 1.75 * 2^8: a mantissa above
// 1.75 carries into the exponent.
__device__ __forceinline__ uint32_t row_exponent(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return kExpNan;
    const uint32_t e = (amax_bits + 0x1fffffu) >> 23;
    return e > 8u ? e - 8u : 0u;
}

// 2^(127 - E), the factor before rounding (E <= 247 for every finite row).
__device__ __forceinline__ float inv_scale(uint32_t E) { return __uint_as_float((254u - E) << 23); }

// 2^(E - 127), the factor of the stored values; NaN for E = 255.
__device__ __forceinline__ float row_scale(uint32_t E) {
    return __uint_as_float(E == 0u ? 0x00400000u : E == kExpNan ? 0x7fc00000u : E << 23);
}

// Two fp32 values to two e4m3 bytes (low byte first), round to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 bytes to an fp16 pair (exact: every e4m3 value is an fp16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

}  // namespace fa
