// fa_cache.cu -- rows written into a paged key/value cache and read back (sm_103a).
//
// fa_cache_append: new_lens[b] key and value rows of sequence b go to its last slots,
// tokens seq_lens[b] - new_lens[b] .. seq_lens[b] - 1; token t lives in page
// block_tables[b][t / 16] at slot t % 16.  Keys may be rotated on the way (rotary positions, the
// token's index being its position); an e4m3 cache gets the row quantised (fa_e4m3.cuh) from
// its fp32 values, a 16-bit cache the 16-bit row.  fa_cache_read gathers the pages of a sequence
// into dense 16-bit rows, zeros past its end.
//
// Both are bound by HBM (a few FLOPs per byte).  A thread owns 16 elements of a row when writing, 8
// when reading; the threads of a block lie along tokens first (consecutive tokens of a head are
// contiguous in a page) and, when a call adds fewer tokens than a block has rows (decoding adds
// one), along heads.  The page lookup and the rotation angles depend on the token only, so a thread
// computes them once and walks over the heads of its chunk.
//
// 8 prompts of 1024 to 2048 tokens, 32 heads of 128, rotated, e4m3: written in 59 us (5.1 TB/s), read
// back in 60 (6.2 TB/s).
#include <type_traits>

#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Reports bad device data (a length or a page index); what has it counts as absent.
__device__ __forceinline__ bool bad_arg(int* status) {
    atomicCAS(status, 0, (int)kDevBadArg);
    return false;
}

// Rows of a block: `1 << log_tok` tokens times the rest along heads.
struct RowMap {
    int log_tok;         // log2 of the tokens per block
    int heads_per_block; // heads that a block walks over
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2<BF16>(w[i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                      pack2<BF16>(x[6], x[7]));
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {  // a NaN operand wins
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// fp32 pattern of the largest magnitude of a row (a NaN's if it holds one) from this thread's 16
// values; the row's threads are the D / 16 lanes around this one.
template <int D>
__device__ __forceinline__ uint32_t row_amax(const float (&a)[8], const float (&b)[8]) {
    float mx = max_nan(fabsf(a[0]), fabsf(b[0]), fabsf(a[1]));
    mx = max_nan(mx, fabsf(b[1]), fabsf(a[2]));
    mx = max_nan(mx, fabsf(b[2]), fabsf(a[3]));
    mx = max_nan(mx, fabsf(b[3]), fabsf(a[4]));
    mx = max_nan(mx, fabsf(b[4]), fabsf(a[5]));
    mx = max_nan(mx, fabsf(b[5]), fabsf(a[6]));
    mx = max_nan(mx, fabsf(b[6]), fabsf(a[7]));
    mx = max_nan(mx, mx, fabsf(b[7]));
#pragma unroll
    for (int off = D / 32; off > 0; off >>= 1)
        mx = max_nan(mx, mx, __shfl_xor_sync(0xffffffffu, mx, off));
    return __float_as_uint(mx) & 0x7fffffffu;
}

// Eight values as e4m3 under the row's exponent.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float f) {
    return make_uint2(e4m3x2(x[0] * f, x[1] * f) | (e4m3x2(x[2] * f, x[3] * f) << 16),
                      e4m3x2(x[4] * f, x[5] * f) | (e4m3x2(x[6] * f, x[7] * f) << 16));
}

// Writes a row's 16 values of this thread (a and b, at elements ea and eb of row `dst`) as e4m3, and
// the row's exponent.  Called by all lanes of a warp.
template <int D>
__device__ __forceinline__ void store_e4m3(uint8_t* dst, uint8_t* exp, int ea, int eb, bool first,
                                           const float (&a)[8], const float (&b)[8], bool live) {
    const uint32_t E = row_exponent(row_amax<D>(a, b));
    const float f = E == kExpNan ? 0.0f : inv_scale(E);
    if (live) {
        *reinterpret_cast<uint2*>(dst + ea) = quantise8(a, f);
        *reinterpret_cast<uint2*>(dst + eb) = quantise8(b, f);
        if (first) *exp = (uint8_t)E;
    }
}

// A thread has two 16-byte units of a row, its key's and its value's: for half pairs on unit
// borders (rotary_dim a multiple of 16) a unit and its partner, so that the turn needs no other
// lane, else two neighbours.  The next head's four loads are in flight while a head is written (and
// the first head's while lengths, page and angles are looked up: whether the row is a new one is
// known only then); with one 16-byte load under way per thread the kernel ran at 2.8 TB/s.
// MODE: how keys are turned: 0 not at all, 1 half pairs on unit borders, 2 interleaved, 3 half pairs
// anywhere.
template <int D, bool BF16, bool Q8, int MODE>
__global__ void __launch_bounds__(kThreads, 3)
    fa_cache_append_kernel(const __grid_constant__ CacheAppendParams p, const RowMap m) {
    constexpr int kTpr = D / 16;              // threads per row, 16 elements each
    constexpr int kRows = kThreads / kTpr;    // rows per block
    const int b = blockIdx.z;
    const int j = threadIdx.x % kTpr, row = threadIdx.x / kTpr;
    const int t = (int)blockIdx.x * (1 << m.log_tok) + (row & ((1 << m.log_tok) - 1));
    const int h_step = kRows >> m.log_tok;
    const int h_lane = row >> m.log_tok;
    const int rd = p.rot.rotary_dim, half = rd / 2;
    int ea = 16 * j, eb = ea + 8;  // this thread's elements
    if (MODE == 1 && 16 * j < rd) {
        ea = 8 * j;
        eb = ea + half;
    }
    const int h_end = min(p.H, ((int)blockIdx.y + 1) * m.heads_per_block);
    const int h_first = (int)blockIdx.y * m.heads_per_block;
    const uint8_t* src_k = static_cast<const uint8_t*>(p.k) + 2 * (b * p.sk.b + t * p.sk.l);
    const uint8_t* src_v = static_cast<const uint8_t*>(p.v) + 2 * (b * p.sv.b + t * p.sv.l);
    uint4 next[4];
    auto load = [&](int h, bool there) {
        if (there && h < h_end) {
            const uint8_t *k = src_k + 2 * (h * p.sk.h), *v = src_v + 2 * (h * p.sv.h);
            next[0] = *reinterpret_cast<const uint4*>(k + 2 * ea);
            next[1] = *reinterpret_cast<const uint4*>(k + 2 * eb);
            next[2] = *reinterpret_cast<const uint4*>(v + 2 * ea);
            next[3] = *reinterpret_cast<const uint4*>(v + 2 * eb);
        }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = make_uint4(0u, 0u, 0u, 0u);
    load(h_first + h_lane, t < p.L);

    const int len = p.seq_lens[b];
    int n_new = p.new_lens ? p.new_lens[b] : (len == 0 ? 0 : p.L);
    if (n_new < 0 || n_new > p.L || len < n_new || len > (long long)p.max_pages * kPageTokens) {
        if (threadIdx.x == 0) bad_arg(p.status);
        n_new = 0;
    }
    // The block's warps leave together when no row of it is new.
    if ((int)blockIdx.x * (1 << m.log_tok) >= n_new) return;
    bool ok = t < n_new;
    const int pos = len - n_new + t;
    int page = 0;
    if (ok) {
        page = p.block_tables[(size_t)b * p.max_pages + pos / kPageTokens];
        if (page < 0 || page >= p.num_pages) ok = bad_arg(p.status);
    }
    const int slot = pos % kPageTokens;

    // Angles: pair i of (a, b) (half pairs), or of a, then of b (interleaved).
    constexpr int kAngles = (MODE == 1 || MODE == 2) ? 8 : 1;
    float c[kAngles], s[kAngles];
    if constexpr (MODE == 1 || MODE == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int f = 8 * j + i;
            c[i] = 1.0f;
            s[i] = 0.0f;
            if (ok && f < half) rope_cos_sin(pos, p.rot.freqs[f], p.rot.mscale, c[i], s[i]);
        }
    }
    // Row of the cache of this token's first head here; heads are kPageTokens rows apart.
    constexpr int kRowBytes = D * (Q8 ? 1 : 2);
    const size_t unit0 = ((size_t)page * p.H + h_first + h_lane) * kPageTokens + slot;
    const size_t step = (size_t)h_step * kPageTokens;
    uint8_t* dst_k = static_cast<uint8_t*>(p.k_cache) + unit0 * kRowBytes;
    uint8_t* dst_v = static_cast<uint8_t*>(p.v_cache) + unit0 * kRowBytes;
    uint8_t *exp_k = p.k_exp + unit0, *exp_v = p.v_exp + unit0;
    // Every lane of a warp takes the same number of steps (the shuffles need all lanes).
    for (int h0 = h_first; h0 < h_end; h0 += h_step) {
        const int h = h0 + h_lane;
        const bool live = ok && h < h_end;
        uint4 raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = next[i];
        load(h + h_step, ok);
        float a[8], bb[8];
        if (Q8 || MODE != 0) {
            unpack8<BF16>(raw[0], a);
            unpack8<BF16>(raw[1], bb);
        }
        if constexpr (MODE == 1) {
            if (16 * j < rd) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = a[i] * c[i] - bb[i] * s[i];
                    bb[i] = bb[i] * c[i] + a[i] * s[i];
                    a[i] = y;
                }
            }
        } else if constexpr (MODE == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (ea + 2 * i < rd) {
                    const float y = a[2 * i] * c[i] - a[2 * i + 1] * s[i];
                    a[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * s[i];
                    a[2 * i] = y;
                }
                if (eb + 2 * i < rd) {
                    const float y = bb[2 * i] * c[i + 4] - bb[2 * i + 1] * s[i + 4];
                    bb[2 * i + 1] = bb[2 * i + 1] * c[i + 4] + bb[2 * i] * s[i + 4];
                    bb[2 * i] = y;
                }
            }
        } else if constexpr (MODE == 3) {
            const uint16_t* row16 = reinterpret_cast<const uint16_t*>(src_k + 2 * (h * p.sk.h));
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const int e = ea + i;
                if (!live || e >= rd) break;
                const bool second = e >= half;
                float cc, ss;
                rope_cos_sin(pos, p.rot.freqs[second ? e - half : e], p.rot.mscale, cc, ss);
                const float mine = unpack2<BF16>(row16[e]).x;
                const float other = unpack2<BF16>(row16[second ? e - half : e + half]).x;
                const float y = mine * cc + (second ? other : -other) * ss;
#pragma unroll
                for (int k = 0; k < 8; ++k) {  // (registers have no index)
                    if (k == i) a[k] = y;
                    if (k + 8 == i) bb[k] = y;
                }
            }
        }
        if constexpr (Q8) {
            store_e4m3<D>(dst_k, exp_k, ea, eb, j == 0, a, bb, live);
            unpack8<BF16>(raw[2], a);
            unpack8<BF16>(raw[3], bb);
            store_e4m3<D>(dst_v, exp_v, ea, eb, j == 0, a, bb, live);
        } else if (live) {
            if (MODE != 0) {
                raw[0] = pack8<BF16>(a);
                raw[1] = pack8<BF16>(bb);
            }
            *reinterpret_cast<uint4*>(dst_k + 2 * ea) = raw[0];
            *reinterpret_cast<uint4*>(dst_k + 2 * eb) = raw[1];
            *reinterpret_cast<uint4*>(dst_v + 2 * ea) = raw[2];
            *reinterpret_cast<uint4*>(dst_v + 2 * eb) = raw[3];
        }
        dst_k += step * kRowBytes;
        dst_v += step * kRowBytes;
        exp_k += step;
        exp_v += step;
    }
}

// A thread's unit is 8 elements: 16 bytes of the output (and 8 or 16 of the cache), so that a warp's
// stores are whole rows; two heads' keys and values are loaded together.  (16 elements per thread,
// in one load and two stores 32 bytes apart, took 72 us where this takes 60.)
template <int D, bool BF16, bool Q8>
__global__ void __launch_bounds__(kThreads)
    fa_cache_read_kernel(const __grid_constant__ CacheReadParams p, const RowMap m) {
    constexpr int kTpr = D / 8;
    constexpr int kRows = kThreads / kTpr;
    const int b = blockIdx.z;
    const int row = threadIdx.x / kTpr, e0 = (threadIdx.x % kTpr) * 8;
    const int t = (int)blockIdx.x * (1 << m.log_tok) + (row & ((1 << m.log_tok) - 1));
    const int h_step = kRows >> m.log_tok;
    const int h_lane = row >> m.log_tok;
    if (t >= p.L) return;
    int len = p.seq_lens[b];
    if (len < 0 || len > (long long)p.max_pages * kPageTokens) {
        bad_arg(p.status);
        len = 0;
    }
    bool live = t < len;
    int page = 0;
    if (live) {
        page = p.block_tables[(size_t)b * p.max_pages + t / kPageTokens];
        if (page < 0 || page >= p.num_pages) live = bad_arg(p.status);
    }
    const int slot = t % kPageTokens;
    const int h_end = min(p.H, ((int)blockIdx.y + 1) * m.heads_per_block);
    using In = typename std::conditional<Q8, uint2, uint4>::type;  // 8 elements of the cache
    const In *kc = static_cast<const In*>(p.k_cache), *vc = static_cast<const In*>(p.v_cache);
    uint8_t* out_k = static_cast<uint8_t*>(p.k) + 2 * (b * p.sk.b + t * p.sk.l + e0);
    uint8_t* out_v = static_cast<uint8_t*>(p.v) + 2 * (b * p.sv.b + t * p.sv.l + e0);
    for (int h = (int)blockIdx.y * m.heads_per_block + h_lane; h < h_end; h += 2 * h_step) {
        In q[4];     // key and value of this head, of the next
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int hh = h + (i >> 1) * h_step;
            if (live && hh < h_end) {
                const size_t unit = ((size_t)page * p.H + hh) * kPageTokens + slot;
                q[i] = ((i & 1) ? vc : kc)[unit * (D / 8) + e0 / 8];
                if constexpr (Q8) f[i] = row_scale(((i & 1) ? p.v_exp : p.k_exp)[unit]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int hh = h + (i >> 1) * h_step;
            if (hh >= h_end) break;
            uint4 out = make_uint4(0u, 0u, 0u, 0u);
            if (live) {
                if constexpr (Q8) {
                    const uint32_t two[4] = {q[i].x & 0xffffu, q[i].x >> 16, q[i].y & 0xffffu, q[i].y >> 16};
                    uint32_t r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 x = unpack2<false>(e4m3x2_to_f16x2(two[k]));
                        r[k] = pack2<BF16>(x.x * f[i], x.y * f[i]);
                    }
                    out = make_uint4(r[0], r[1], r[2], r[3]);
                } else {
                    out = q[i];
                }
            }
            uint8_t* dst = (i & 1) ? out_v + 2 * (hh * p.sv.h) : out_k + 2 * (hh * p.sk.h);
            *reinterpret_cast<uint4*>(dst) = out;
        }
    }
}

constexpr int kMaxHeadsPerBlock = 8;

// Tokens per block: a power of two up to the block's rows that covers L.  Heads per block: up to
// kMaxHeadsPerBlock, fewer while the grid has under four blocks per SM.  (2, 4, 8, 16, 32 heads: the
// prompts above take 137, 124, 121, 122, 122 us when the writing has them, 126, 122, 121, 125, 136 when
// the reading has.)
bool row_map(int B, int H, int L, int rows, RowMap* m, dim3* grid) {
    m->log_tok = 0;
    while ((1 << m->log_tok) < rows && (1 << m->log_tok) < L) ++m->log_tok;
    const int tok = 1 << m->log_tok, h_step = rows / tok;
    const int sms = sm_count() > 0 ? sm_count() : 152;
    const long long tiles = ((long long)L + tok - 1) / tok;
    int per = kMaxHeadsPerBlock > h_step ? kMaxHeadsPerBlock : h_step;
    while (per > h_step && tiles * B * ((H + per - 1) / per) < 4LL * sms) per /= 2;
    if (per < h_step) per = h_step;
    m->heads_per_block = per;
    *grid = dim3((unsigned)tiles, (unsigned)((H + per - 1) / per), (unsigned)B);
    return grid->y <= 65535u && B <= 65535;
}

}  // namespace

namespace {
template <int D, bool BF16, bool Q8>
cudaError_t launch_append(const CacheAppendParams& p, cudaStream_t s) {
    RowMap m;
    dim3 grid;
    if (!row_map(p.B, p.H, p.L, kThreads / (D / 16), &m, &grid))
        return cudaErrorInvalidConfiguration;
    auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(kThreads), 0, s, p, m); };
    if (p.rot.rotary_dim == 0) return go(fa_cache_append_kernel<D, BF16, Q8, 0>);
    if (p.rot.interleaved) return go(fa_cache_append_kernel<D, BF16, Q8, 2>);
    return p.rot.rotary_dim % 16 == 0 ? go(fa_cache_append_kernel<D, BF16, Q8, 1>)
                                      : go(fa_cache_append_kernel<D, BF16, Q8, 3>);
}
template <int D, bool BF16>
cudaError_t launch_append_q(const CacheAppendParams& p, bool q8, cudaStream_t s) {
    return q8 ? launch_append<D, BF16, true>(p, s) : launch_append<D, BF16, false>(p, s);
}
}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, bool bf16, bool q8, cudaStream_t s) {
    if (p.D == 64) return bf16 ? launch_append_q<64, true>(p, q8, s) : launch_append_q<64, false>(p, q8, s);
    return bf16 ? launch_append_q<128, true>(p, q8, s) : launch_append_q<128, false>(p, q8, s);
}

cudaError_t launch_cache_read(const CacheReadParams& p, bool bf16, bool q8, cudaStream_t s) {
    RowMap m;
    dim3 grid;
    if (!row_map(p.B, p.H, p.L, kThreads / (p.D / 8), &m, &grid)) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(kThreads), 0, s, p, m); };
    if (q8)
        return p.D == 64 ? (bf16 ? go(fa_cache_read_kernel<64, true, true>)
                                 : go(fa_cache_read_kernel<64, false, true>))
                         : (bf16 ? go(fa_cache_read_kernel<128, true, true>)
                                 : go(fa_cache_read_kernel<128, false, true>));
    return p.D == 64 ? (bf16 ? go(fa_cache_read_kernel<64, true, false>)
                             : go(fa_cache_read_kernel<64, false, false>))
                     : (bf16 ? go(fa_cache_read_kernel<128, true, false>)
                             : go(fa_cache_read_kernel<128, false, false>));
}

}  // namespace fa
