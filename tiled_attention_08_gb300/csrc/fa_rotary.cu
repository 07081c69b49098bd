// fa_rotary.cu -- rotary positions on queries and keys, both directions (sm_103a).
//
// Row l of sequence b at position m: each pair (x1, x2) of the first rotary_dim elements becomes
//     y1 = mscale (x1 cos(m theta_i) - x2 sin(m theta_i)),
//     y2 = mscale (x2 cos(m theta_i) + x1 sin(m theta_i)),
// pairs being (i, i + rotary_dim/2) or, interleaved, (2i, 2i+1); the other elements pass through.
// The map is linear and orthogonal up to mscale, so the gradient is the same kernel with the
// sign of the angle flipped (`inverse`).
//
// Bound by HBM: 4 bytes moved per element against 3 FLOPs.  The angles are the only arithmetic
// of weight (per pair one 64-bit product and a sine and cosine), and they are the same for every
// head of a token: a thread owns 8 or 16 elements of one token (one 16-byte unit, or the unit
// and its partner rotary_dim/2 away), computes their angles once and walks over the heads of
// its chunk, four heads' loads in flight at a time.  Queries and keys share one launch: their
// heads form one list.  Work in place is safe, since each element is read and written by the
// same thread.
//
// 8 x 4096 tokens, 32 + 32 heads of 128, bf16: 160 us (6.7 TB/s, 99% of a copy's rate), in either
// direction; 256 tokens of a decode batch, 32 + 8 heads: 4.5 us, a launch.
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2<BF16>(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                      pack2<BF16>(f[6], f[7]));
}

__device__ __forceinline__ int token_position(const RotaryLaunch& p, long long b, int l) {
    return p.positions ? p.positions[b * p.pos_stride + l] : l;
}

// 16-byte units.  Half pairs (rotary_dim a multiple of 16): unit u < rotary_dim/16 is the
// elements 8u.. and their partners rotary_dim/2 further, a unit after them 16 elements to copy.
// Interleaved (rotary_dim a multiple of 8): unit u is the elements 8u.., copied from
// u = rotary_dim/8 on.  Turned and copied units take the same path (the copy returns what it
// loaded), since both lie in one warp.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_rotary_kernel(const RotaryLaunch p, int units,
                                                             int heads_per_block) {
    constexpr int kUnroll = 4;
    const int rd = p.rot.rotary_dim;
    const int n_rot = INTER ? rd / 8 : rd / 16;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long token = id / units;
    const int u = (int)(id - token * units);
    if (token >= (long long)p.B * p.L) return;
    const long long b = token / p.L;
    const int l = (int)(token - b * p.L);
    const int heads = p.op[0].H + p.op[1].H;
    const int h0 = (int)blockIdx.y * heads_per_block;
    const int h1 = min(heads, h0 + heads_per_block);
    const bool turn = u < n_rot;
    // Byte offsets of the unit and, for half pairs, of its second 16 bytes.
    const int lo = (INTER || turn) ? u * 16 : rd * 2 + (u - n_rot) * 32;
    const int hi = turn ? lo + rd : lo + 16;
    auto source = [&](int h) {
        const RotaryOperand& o = p.op[h < p.op[0].H ? 0 : 1];
        const int hh = h < p.op[0].H ? h : h - p.op[0].H;
        return static_cast<const uint8_t*>(o.x) + 2 * (b * o.sx.b + hh * o.sx.h + l * o.sx.l);
    };
    uint4 xa[kUnroll], xb[kUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (h + j >= h1) break;
            const uint8_t* src = source(h + j);
            xa[j] = *reinterpret_cast<const uint4*>(src + lo);
            if (!INTER) xb[j] = *reinterpret_cast<const uint4*>(src + hi);
        }
    };
    load(h0);  // in flight while the angles are computed
    constexpr int kPairs = INTER ? 4 : 8;
    float c[kPairs], s[kPairs];
    if (turn) {
        const int pos = token_position(p, b, l);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            rope_cos_sin(pos, p.rot.freqs[u * kPairs + i], p.rot.mscale, c[i], s[i]);
            if (p.inverse) s[i] = -s[i];
        }
    }
    for (int h = h0; h < h1; h += kUnroll) {
        if (h > h0) load(h);
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (h + j >= h1) break;
            uint4 ya = xa[j], yb = xb[j];
            if (turn) {
                float a[8], y[8];
                unpack8<BF16>(xa[j], a);
                if constexpr (INTER) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[2 * i] = a[2 * i] * c[i] - a[2 * i + 1] * s[i];
                        y[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * s[i];
                    }
                } else {
                    float bb[8], z[8];
                    unpack8<BF16>(xb[j], bb);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] = a[i] * c[i] - bb[i] * s[i];
                        z[i] = bb[i] * c[i] + a[i] * s[i];
                    }
                    yb = pack8<BF16>(z);
                }
                ya = pack8<BF16>(y);
            }
            const RotaryOperand& o = p.op[h + j < p.op[0].H ? 0 : 1];
            const int hh = h + j < p.op[0].H ? h + j : h + j - p.op[0].H;
            uint8_t* dst = static_cast<uint8_t*>(o.y) + 2 * (b * o.sy.b + hh * o.sy.h + l * o.sy.l);
            *reinterpret_cast<uint4*>(dst + lo) = ya;
            if (!INTER) *reinterpret_cast<uint4*>(dst + hi) = yb;
        }
    }
}

// Any even rotary_dim (pairs that do not fall on 16-byte units): one pair, or one element past
// rotary_dim, per thread and head.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_rotary_pairs_kernel(const RotaryLaunch p, int units,
                                                                   int heads_per_block) {
    const int rd = p.rot.rotary_dim;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long token = id / units;
    const int u = (int)(id - token * units);
    if (token >= (long long)p.B * p.L) return;
    const long long b = token / p.L;
    const int l = (int)(token - b * p.L);
    const int heads = p.op[0].H + p.op[1].H;
    const int h0 = (int)blockIdx.y * heads_per_block;
    const int h1 = min(heads, h0 + heads_per_block);
    const bool pair = u < rd / 2;
    float c = 1.0f, s = 0.0f;
    if (pair) rope_cos_sin(token_position(p, b, l), p.rot.freqs[u], p.rot.mscale, c, s);
    if (p.inverse) s = -s;
    const int ia = pair ? (INTER ? 2 * u : u) : rd / 2 + u;
    const int ib = INTER ? ia + 1 : ia + rd / 2;
    for (int h = h0; h < h1; ++h) {
        const RotaryOperand& o = p.op[h < p.op[0].H ? 0 : 1];
        const int hh = h < p.op[0].H ? h : h - p.op[0].H;
        const uint16_t* src =
            static_cast<const uint16_t*>(o.x) + b * o.sx.b + hh * o.sx.h + l * o.sx.l;
        uint16_t* dst = static_cast<uint16_t*>(o.y) + b * o.sy.b + hh * o.sy.h + l * o.sy.l;
        if (!pair) {
            dst[ia] = src[ia];
            continue;
        }
        const float2 x = unpack2<BF16>((uint32_t)src[ia] | ((uint32_t)src[ib] << 16));
        const uint32_t y = pack2<BF16>(x.x * c - x.y * s, x.y * c + x.x * s);
        dst[ia] = (uint16_t)(y & 0xffffu);
        dst[ib] = (uint16_t)(y >> 16);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& p, bool bf16, cudaStream_t s) {
    const int rd = p.rot.rotary_dim, inter = p.rot.interleaved;
    const bool vec = rd % (inter ? 8 : 16) == 0;
    const int n_rot = vec ? (inter ? rd / 8 : rd / 16) : rd / 2;
    const int units = n_rot + (p.copy_rest ? (vec ? (p.D - rd) / (inter ? 8 : 16) : p.D - rd) : 0);
    const long long blocks = ((long long)p.B * p.L * units + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int heads = p.op[0].H + p.op[1].H;
    // Heads per block: as many as leave about eight blocks per SM (the angles are shared by
    // more heads), at most 16.
    const int sms = sm_count() > 0 ? sm_count() : 152;
    int per = 16;
    while (per > 1 && blocks * ((heads + per - 1) / per) < 8LL * sms) per /= 2;
    const dim3 grid((unsigned)blocks, (unsigned)((heads + per - 1) / per));
    if (grid.y > 65535u) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(kThreads), 0, s, p, units, per); };
    if (vec)
        return bf16 ? (inter ? go(fa_rotary_kernel<true, true>) : go(fa_rotary_kernel<true, false>))
                    : (inter ? go(fa_rotary_kernel<false, true>) : go(fa_rotary_kernel<false, false>));
    return bf16 ? (inter ? go(fa_rotary_pairs_kernel<true, true>)
                         : go(fa_rotary_pairs_kernel<true, false>))
                : (inter ? go(fa_rotary_pairs_kernel<false, true>)
                         : go(fa_rotary_pairs_kernel<false, false>));
}

}  // namespace fa
