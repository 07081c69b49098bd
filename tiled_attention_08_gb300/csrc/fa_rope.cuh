// fa_rope.cuh -- the rotation angles of rotary positions (device helpers).
#pragma once

#include <stdint.h>

namespace fa {

// cos and sin of position * theta, times mscale.  theta is held in turns per position as a
// 64-bit fixed-point fraction (freq = theta / (2 pi) * 2^64), so the wrapped 64-bit product
// position * freq is the angle reduced modulo one turn, exactly: for |position| < 2^31 the error
// left is that of freq's rounding, under 2^-33 turns, where a 32-bit product would have lost
// 2^-24 of up to 2^31 radians.  Its top 32 bits, as a signed fraction of a turn in [-1/2, 1/2),
// become an fp32 angle in [-pi, pi] (relative error 2^-23), where the hardware's sine and cosine
// are within 2^-21: far below half a step of the 16-bit (2^-9, 2^-12) and 8-bit results.
__device__ __forceinline__ void rope_cos_sin(int position, long long freq, float mscale, float& c,
                                             float& s) {
    const long long turns = (long long)position * freq;  // wraps modulo one turn
    const float a = (float)(int)(turns >> 32) * 1.4629180792671596e-09f;  // 2 pi / 2^32
    __sincosf(a, &s, &c);
    c *= mscale;
    s *= mscale;
}

}  // namespace fa
