// fa_rope.cuh -- the rotation angles of rotary positions (device helpers).
#pragma once

#include <stdint.h>

namespace fa {

// cos and sin of position * theta, times mscale.  theta is held in turns per position as a
// 64-bit fixed-point fraction (freq = theta / (2 pi) * 2^64), so the wrapped 64-bit product
// position * freq is the angle reduced modulo one turn, exactly.  The error left is that of the
// table, whose theta is good to a few units of 2^-53 (an fp64 power and quotient) and so moves the
// angle by |position| times that (2^-32 of theta's turns at position 2^20, 2^-21 at 2^31), and 2^-32
// turns for the bits below the upper half; a 32-bit product would have lost 2^-24 of the whole
// angle.  The nearest quarter turn is split off in integers too, so that
// the rest, at most an eighth of a turn, becomes an fp32 with an error of 2^-27 half turns.  The
// hardware's sine and cosine (2^-21) would do for 16-bit results, but move eight times as many
// values of an 8-bit cache over a rounding border as fp32's own rounding; sincospif costs a
// few more instructions per angle, which all heads of a token share.
__device__ __forceinline__ void rope_cos_sin(int position, long long freq, float mscale, float& c,
                                             float& s) {
    const uint32_t turns = (uint32_t)(((long long)position * freq) >> 32);  // 2^32 = one turn
    const uint32_t quarter = (turns + 0x20000000u) >> 30;
    float sn, cs;
    sincospif((float)(int)(turns - (quarter << 30)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
    c = ((quarter & 1u) ? sn : cs) * mscale;
    s = ((quarter & 1u) ? cs : sn) * mscale;
    if (((quarter + 1u) & 2u)) c = -c;  // quarters 1 and 2
    if (quarter & 2u) s = -s;           // quarters 2 and 3
}

}  // namespace fa
