// fa_cache.cu -- rows written into a paged key/value cache and read back (sm_103a).
//
// fa_cache_append: new_lens[b] key and value rows of sequence b go to its last slots,
// tokens seq_lens[b] - new_lens[b] .. seq_lens[b] - 1; token t lives in page
// block_tables[b][t / 16] at slot t % 16.  Keys may be rotated on the way (rotary positions, the
// token's index being its position); an e4m3 cache gets the row quantised (fa_e4m3.cuh) from
// its fp32 values, a 16-bit cache the 16-bit row.  fa_cache_read gathers the pages of a sequence
// into dense 16-bit rows, zeros past its end.
//
// Both are bound by HBM (a few FLOPs per byte).  A thread owns one 16-byte unit of a row; the
// threads of a block lie along tokens first (consecutive tokens of a head are contiguous in a
// page) and, when a call adds fewer tokens than a block has rows (decoding adds one), along heads.
// The page lookup and the rotation angles depend on the token only, so a thread computes them
// once and walks over the heads of its chunk.
#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Checks a sequence's length against the table; a bad one counts as empty and is reported.
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

// Writes this thread's 8 elements of a row (its values x, or the 16-bit ones it was given) to
// row `unit` of a cache; the row's threads are the kTpr lanes around this one.
template <int D, bool BF16, bool Q8>
__device__ __forceinline__ void store_unit(void* cache, uint8_t* exps, size_t unit, int chunk,
                                           const float (&x)[8], const uint4& raw, bool live) {
    if constexpr (Q8) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int off = D / 16; off > 0; off >>= 1)
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const uint32_t E = row_exponent(mx);
        const float f = E == kExpNan ? 0.0f : inv_scale(E);
        if (live) {
            uint2 q;
            q.x = e4m3x2(x[0] * f, x[1] * f) | (e4m3x2(x[2] * f, x[3] * f) << 16);
            q.y = e4m3x2(x[4] * f, x[5] * f) | (e4m3x2(x[6] * f, x[7] * f) << 16);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + unit * D + chunk * 8) = q;
            if (chunk == 0) exps[unit] = (uint8_t)E;
        }
    } else if (live) {
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(cache) + (unit * D + chunk * 8) * 2) = raw;
    }
}

// The loads of the next head's key and value are in flight while a head is worked on (and the
// first head's while lengths, page and angles are looked up: whether the row is a new one is
// known only then).  Without that each thread had one 16-byte load under way and the kernel ran at
// 2.8 TB/s.
template <int D, bool BF16, bool Q8>
__global__ void __launch_bounds__(kThreads, 3)
    fa_cache_append_kernel(const __grid_constant__ CacheAppendParams p, const RowMap m) {
    constexpr int kTpr = D / 8;               // threads per row, 8 elements each
    constexpr int kRows = kThreads / kTpr;    // rows per block
    const int b = blockIdx.z;
    const int chunk = threadIdx.x % kTpr, row = threadIdx.x / kTpr;
    const int t = (int)blockIdx.x * (1 << m.log_tok) + (row & ((1 << m.log_tok) - 1));
    const int h_step = kRows >> m.log_tok;
    const int h_lane = row >> m.log_tok;
    const int e0 = chunk * 8;
    const int h_end = min(p.H, ((int)blockIdx.y + 1) * m.heads_per_block);
    const int h_first = (int)blockIdx.y * m.heads_per_block;
    const uint8_t* src_k = static_cast<const uint8_t*>(p.k) + 2 * (b * p.sk.b + t * p.sk.l + e0);
    const uint8_t* src_v = static_cast<const uint8_t*>(p.v) + 2 * (b * p.sv.b + t * p.sv.l + e0);
    auto load = [&](const uint8_t* src, long long stride, int h, bool there) {
        return there && h < h_end ? *reinterpret_cast<const uint4*>(src + 2 * (h * stride))
                                  : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 next_k = load(src_k, p.sk.h, h_first + h_lane, t < p.L);
    uint4 next_v = load(src_v, p.sv.h, h_first + h_lane, t < p.L);

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

    // This thread's rotation: element i of its unit and its partner, y = x c + partner s.
    const int rd = p.rot.rotary_dim, half = rd / 2;
    const bool inter = p.rot.interleaved != 0;
    float c[8], s[8];
    if (rd > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            c[i] = 1.0f;
            s[i] = 0.0f;
            if (inter && (i & 1)) {  // the pair's second element: the same angle
                c[i] = c[i - 1];
                s[i] = -s[i - 1];
            } else if (ok && e < rd) {
                const int f = inter ? e >> 1 : (e < half ? e : e - half);
                rope_cos_sin(pos, p.rot.freqs[f], p.rot.mscale, c[i], s[i]);
                if (inter || e < half) s[i] = -s[i];
            }
        }
    }
    // Lane of the unit that holds the partners of half pairs (rotary_dim a multiple of 16).
    const int d = rd / 16;
    const int partner = (threadIdx.x & 31) + (e0 < half ? d : (e0 < rd ? -d : 0));
    // Every lane of a warp takes the same number of steps (the shuffles need all lanes).
    for (int h0 = h_first; h0 < h_end; h0 += h_step) {
        const int h = h0 + h_lane;
        const bool live = ok && h < h_end;
        uint4 raw_k = next_k;
        const uint4 raw_v = next_v;
        next_k = load(src_k, p.sk.h, h + h_step, ok);
        next_v = load(src_v, p.sv.h, h + h_step, ok);
        const size_t unit = ((size_t)page * p.H + h) * kPageTokens + slot;  // row of the cache
        float x[8];
        unpack8<BF16>(raw_k, x);
        if (rd > 0) {
            float o[8];  // the partners
            if (inter) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
            } else if (rd % 16 == 0) {
                uint4 r;
                r.x = __shfl_sync(0xffffffffu, raw_k.x, partner);
                r.y = __shfl_sync(0xffffffffu, raw_k.y, partner);
                r.z = __shfl_sync(0xffffffffu, raw_k.z, partner);
                r.w = __shfl_sync(0xffffffffu, raw_k.w, partner);
                unpack8<BF16>(r, o);
            } else {  // pairs that do not fall on 16-byte units
                const uint16_t* row16 = reinterpret_cast<const uint16_t*>(src_k + 2 * (h * p.sk.h)) - e0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = e0 + i;
                    const int q = e < half ? e + half : (e < rd ? e - half : e);
                    o[i] = live ? unpack2<BF16>(row16[q]).x : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i < rd) x[i] = x[i] * c[i] + o[i] * s[i];
            if constexpr (!Q8)
                raw_k = make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]),
                                   pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
        }
        store_unit<D, BF16, Q8>(p.k_cache, p.k_exp, unit, chunk, x, raw_k, live);
        unpack8<BF16>(raw_v, x);
        store_unit<D, BF16, Q8>(p.v_cache, p.v_exp, unit, chunk, x, raw_v, live);
    }
}

// A thread's unit is 8 elements: 16 bytes of the output (8 bytes of an e4m3 cache).
template <int D, bool BF16, bool Q8>
__global__ void __launch_bounds__(kThreads)
    fa_cache_read_kernel(const __grid_constant__ CacheReadParams p, const RowMap m) {
    constexpr int kTpr = D / 8;
    constexpr int kRows = kThreads / kTpr;
    const int b = blockIdx.z;
    const int chunk = threadIdx.x % kTpr, row = threadIdx.x / kTpr;
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
    const int slot = t % kPageTokens, e0 = chunk * 8;
    const int h_end = min(p.H, ((int)blockIdx.y + 1) * m.heads_per_block);
    for (int h = (int)blockIdx.y * m.heads_per_block + h_lane; h < h_end; h += h_step) {
        const size_t unit = ((size_t)page * p.H + h) * kPageTokens + slot;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint8_t* src = static_cast<const uint8_t*>(which ? p.v_cache : p.k_cache);
            uint4 out = make_uint4(0u, 0u, 0u, 0u);
            if (live) {
                if constexpr (Q8) {
                    const uint2 q = *reinterpret_cast<const uint2*>(src + unit * D + e0);
                    const float f = row_scale((which ? p.v_exp : p.k_exp)[unit]);
                    const uint32_t two[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
                    uint32_t r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = unpack2<false>(e4m3x2_to_f16x2(two[i]));
                        r[i] = pack2<BF16>(x.x * f, x.y * f);
                    }
                    out = make_uint4(r[0], r[1], r[2], r[3]);
                } else {
                    out = *reinterpret_cast<const uint4*>(src + (unit * D + e0) * 2);
                }
            }
            const Strides& st = which ? p.sv : p.sk;
            uint8_t* dst = static_cast<uint8_t*>(which ? p.v : p.k) +
                           2 * (b * st.b + h * st.h + t * st.l);
            *reinterpret_cast<uint4*>(dst + e0 * 2) = out;
        }
    }
}

// Tokens per block: a power of two up to the block's rows that covers L.  Heads per block: up to
// `most`, fewer while the grid has under four blocks per SM.
bool row_map(int B, int H, int L, int D, int most, RowMap* m, dim3* grid) {
    const int rows = kThreads / (D / 8);
    m->log_tok = 0;
    while ((1 << m->log_tok) < rows && (1 << m->log_tok) < L) ++m->log_tok;
    const int tok = 1 << m->log_tok, h_step = rows / tok;
    const int sms = sm_count() > 0 ? sm_count() : 152;
    const long long tiles = ((long long)L + tok - 1) / tok;
    int per = most > h_step ? most : h_step;
    while (per > h_step && tiles * B * ((H + per - 1) / per) < 4LL * sms) per /= 2;
    if (per < h_step) per = h_step;
    m->heads_per_block = per;
    *grid = dim3((unsigned)tiles, (unsigned)((H + per - 1) / per), (unsigned)B);
    return grid->y <= 65535u && B <= 65535;
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, bool bf16, bool q8, cudaStream_t s) {
    RowMap m;
    dim3 grid;
    if (!row_map(p.B, p.H, p.L, p.D, 8, &m, &grid)) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(kThreads), 0, s, p, m); };
    if (q8)
        return p.D == 64 ? (bf16 ? go(fa_cache_append_kernel<64, true, true>)
                                 : go(fa_cache_append_kernel<64, false, true>))
                         : (bf16 ? go(fa_cache_append_kernel<128, true, true>)
                                 : go(fa_cache_append_kernel<128, false, true>));
    return p.D == 64 ? (bf16 ? go(fa_cache_append_kernel<64, true, false>)
                             : go(fa_cache_append_kernel<64, false, false>))
                     : (bf16 ? go(fa_cache_append_kernel<128, true, false>)
                             : go(fa_cache_append_kernel<128, false, false>));
}

cudaError_t launch_cache_read(const CacheReadParams& p, bool bf16, bool q8, cudaStream_t s) {
    RowMap m;
    dim3 grid;
    if (!row_map(p.B, p.H, p.L, p.D, 8, &m, &grid)) return cudaErrorInvalidConfiguration;
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
