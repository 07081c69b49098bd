// fa_chunk.cu -- attention of a chunk of new tokens of every sequence over a paged cache (sm_103a).
//
// Sequence b of len_b cached tokens adds its last n_b; row i < n_b of q[b, h] is token len_b - n_b + i
// and attends, causally, to the cached rows of head h / G, all of them or those of a sliding window and
// the first tokens (fa_window_sched.h):  O = softmax(scale q K^T) V and LSE.  Rows i >= n_b get 0, -inf.
//
// 4 G D FLOPs per token pair and cache head: bound by the tensor cores from a few hundred query rows per
// cache head on, by HBM or latency below.  The pipeline is that of the dense forward: two 128-row query
// tiles share every 128-key tile; producer warps, one MMA warp, eight softmax warps (a row per
// thread), P as the TMEM operand of PV.  What differs:
//  * rows: row r of a tile is token r % T of head r / T of the group, T = 128 / G tokens: short chunks
//    fill the tensor core with the group's heads, and each cached row is read once for all of them.  One
//    4-D TMA box {64, T, G, 1} of q brings them in that order.  Rows behind T G hold whatever the slot
//    held: tensor-core rows do not mix, and they are not written.
//  * keys: a 128-key tile is 8 pages.  Of a 16-bit cache each is its own TMA box, issued by one lane
//    each; pages without a token that the pair sees are read at a row outside the map, as zeros, and
//    slots of other pages that hold none are cleared in V by the MMA warp (0 * NaN).  Of an e4m3 cache
//    eight converter warps read the bytes, multiply by the row's power of two in fp32, round to q's type
//    (exact in bf16) and write the tile in the swizzled layout that the contraction reads.
//  * split: lengths are known on the device only, and rows alone seldom fill 152 SMs.  Units (head, pair of
//    query tiles, key tile) form one line, of which every CTA takes an equal stretch: each CTA first
//    sums the pairs' key tiles.  A pair that lies whole in a stretch is written as O and LSE; of a cut
//    one each CTA leaves an fp32 part (two at most), and the one that finds the others' there joins them.  (A kernel
//    of its own for that took 16 of 177 us for the two prompts below, 6 of 24 for one short turn.)
// Measured, this kernel alone: prompts of 2048 and 4096 tokens, 32 heads of 128, 163 us (1060 TFLOP/s); four chunks of
// 1024 to 2048 under a window of 4096, 32 heads on 8, 295 us (1320); eight of 256 to 512 behind 512 to 16384 tokens, 64
// heads on 8, e4m3, 790 us (1240); 17 of 63 to 127 tokens, 16 heads on 4 of 64, 47 us.  A CTA's start (lengths, line,
// first tiles) is 4 us, a cut pair 6 to 13 us.
// Chunks of very few rows per cache head are the decode kernel's (fa_decode_gqa.cu, kRows; few_rows in fa_serve.cu).
#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_window_sched.h"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;
// fp16 weights are taken relative to a reference 2^7 below the largest (see fa_decode_gqa.cu).
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;
constexpr int kPagesPerTile = kTileRows / kPageTokens;

template <int D, bool BF16, bool Q8>
struct ChunkCfg {
    static constexpr int kChunks = D / kChunkElems;
    static constexpr int kTileBytes = kTileRows * D * 2;
    // Tile slots.  16-bit caches: a ring for K and one for V.  e4m3: one ring, K and V in turn, of three
    // slots at D = 128 (a step reads V_j and K_{j+1} while V_{j+1} is converted), which leaves room for
    // 64 KB of bytes in flight, not 32.
    static constexpr int kStages = (D == 128) ? 2 : 4;
    static constexpr int kSlots = Q8 ? ((D == 128) ? 3 : 6) : 2 * kStages;
    static constexpr int kOffQ = 0;
    static constexpr int kOffKV = kOffQ + 2 * kTileBytes;
    // The slot of K (v = 0) or V (v = 1) of the g-th tile, and the how-manieth use of it that is.
    __host__ __device__ static constexpr int slot(int g, int v) {
        return Q8 ? (2 * g + v) % kSlots : v * kStages + g % kStages;
    }
    __host__ __device__ static constexpr int use(int g, int v) { return Q8 ? (2 * g + v) / kSlots : g / kStages; }
    // e4m3: tiles as bytes on their way to the converters, a ring each of K and V, 64 KB in all, and their
    // exponents.
    static constexpr int kRawBytes = kTileRows * D;
    static constexpr int kRaw = Q8 ? 32768 / kRawBytes : 0;
    static constexpr int kOffRaw = kOffKV + kSlots * kTileBytes;
    static constexpr int kOffExp = kOffRaw + 2 * kRaw * kRawBytes;
    static constexpr int kSmemBytes = kOffExp + 2 * kRaw * kTileRows + 1024;
    // 16-bit: the K warp works the segments out and leaves them in a ring of this many.  Done by every warp for itself
    // that took 3000 of the 10000 cycles of an item of one tile (its code is cold whenever it is reached): 309 -> 295 us
    // for the chunks of up to 2048 above, 167.5 -> 163.4 for the prompts.  (e4m3: 92 -> 86 us for 64 chunks of 10 to
    // 20, but 788 -> 817 for the eight of up to 512, whose loops fill the instruction cache; every warp for itself.)
    static constexpr int kSegs = Q8 ? 1 : 4;
    // Warp 8: queries and K; 9: V; 10: MMA; 12 .. 19: converters.
    static constexpr int kKWarp = 8, kVWarp = 9, kMmaWarp = 10, kConvWarp = 12;
    static constexpr int kConverters = Q8 ? 8 : 0;
    static constexpr int kThreads = (Q8 ? 12 + kConverters : 11) * 32;
    // e4m3: registers per thread of the softmax warps and of the others.  At launch each thread has kRegs; the
    // sums over the warpgroups are the same.  (16-bit: 168 for everyone; 208 and 88 took 2% more.)  The
    // e4m3 instances store 596 to 624 bytes of spills a thread, most of them in the softmax warps' loop (248 and 160
    // are left without it, 484 and 520 without the converters'); 16-bit ones 48.
    static constexpr int kRegs = 96, kRegsSoftmax = 168, kRegsOther = 48;
    static_assert(!Q8 || 2 * kRegsSoftmax + (kThreads / 128 - 2) * kRegsOther == kThreads / 128 * kRegs,
                  "the launch's registers");
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kTmS = 0, kTmO = 256;
    static_assert(kTmO + 2 * D <= kTmemCols, "TMEM budget");
    static_assert(kSmemBytes <= 232448 - 768, "shared memory over the 227 KB per-block limit");
    static constexpr uint32_t kIdescS = idesc_f16(BF16, 128, 128, false, false);
    static constexpr uint32_t kIdescO = idesc_f16(BF16, 128, D, false, true);
};

// Every lane of a warp holds a row's 128 bytes, 8 units of 16, bound for dst (null: not written).  The units
// are transposed in groups of eight lanes (a butterfly of xor shuffles; see tmem_rows_to_global_xpose), so that
// each store instruction writes 128 contiguous bytes of four rows.
__device__ __forceinline__ void rows_out(uint32_t (&m)[8][4], uint8_t* dst, int lane) {
#pragma unroll
    for (int s = 4; s >= 1; s /= 2) {
        const bool upper = (lane & s) != 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e & s) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t send = upper ? m[e][k] : m[e | s][k];
                const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, s);
                if (upper) m[e][k] = recv;
                else m[e | s][k] = recv;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // unit lane % 8 of row 8 (lane / 8) + e
        uint8_t* d = reinterpret_cast<uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), (lane & 24) + e));
        if (d)
            *reinterpret_cast<uint4*>(d + (lane & 7) * 16) = make_uint4(m[e][0], m[e][1], m[e][2], m[e][3]);
    }
}

// Sixteen e4m3 bytes times an fp32 power of two, rounded once to 16 bits.  By way of fp16 and fp32: five
// instructions per two values, over the conversion, fp and integer pipes.  (Moving sign, exponent and mantissa to
// their places in bf16 and one 16-bit product are as many, most of them on the integer pipe, and lose a NaN byte and
// rows of extreme size, which then have to be looked for: 792 and 829 us against 774 for the eight chunks of up to 512
// above.)
template <bool BF16>
__device__ __forceinline__ void scaled16(const uint4& x, uint64_t f2, uint32_t (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(h[0]), "=r"(h[1])
            : "r"(w[i]));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 a = unpack2<false>(h[k]);
            float lo, hi;
            f2_split(f2_mul(f2_make(a.x, a.y), f2), lo, hi);
            y[2 * i + k] = pack2<BF16>(lo, hi);
        }
    }
}

// New tokens of sequence b and the tokens in front of them; none where the lengths are out of range.
__device__ __forceinline__ bool sequence(const ChunkParams& p, int b, int& n, int& before) {
    const int len = p.seq_lens[b];
    n = p.new_lens ? p.new_lens[b] : (len > 0 ? p.L : 0);
    before = len - n;
    const bool ok = len >= 0 && len <= (long long)p.max_pages * kPageTokens && n >= 0 && n <= p.L && n <= len &&
                    (n == 0 || p.num_pages > 0);
    if (!ok) n = before = 0;
    return ok;
}
__device__ __forceinline__ int pairs_of(const ChunkParams& p, int n) { return (n + 2 * p.T - 1) / (2 * p.T); }

// Pair i of a sequence: tokens 2 T i .. of its new ones.
__device__ __forceinline__ KeyTiles pair_tiles(const ChunkParams& p, int n, int before, int i) {
    const int t0 = 2 * p.T * i;
    return key_tiles(before + t0, before + imin(t0 + 2 * p.T, n) - 1, p.window, p.sinks);
}

// A place on the line of units and how many of this CTA's lie from there on.
struct Walk {
    int hk, b, pair, j;
    int left;
};

// Key tiles j0 .. j0 + n - 1 (of those of `all`) of a pair of query tiles.
struct Segment {
    int b, hk, t0;         // first new token of the pair
    int fresh, before;     // new tokens of the sequence, tokens in front of them
    KeyTiles all;
    int n_all, j0, n;
    int a_end, b_0, b_1;   // A sees tiles j < a_end of `all`, B those of j < b_0 and j >= b_1
    int done;              // units of the CTA in front of it
    bool has_b;
    __device__ __forceinline__ bool active(int t, int j) const { return t ? has_b && (j < b_0 || j >= b_1) : j < a_end; }
    __device__ __forceinline__ int count(int t) const {  // of the segment's
        const int e = j0 + n;
        if (t == 0) return imax(imin(e, a_end) - j0, 0);
        return has_b ? imax(imin(e, b_0) - j0, 0) + imax(e - imax(j0, b_1), 0) : 0;
    }
    __device__ __forceinline__ bool whole() const { return n == n_all; }
};

__device__ __forceinline__ bool segment_at(const ChunkParams& p, const Walk& w, Segment& s) {
    if (w.left <= 0) return false;
    s.b = w.b;
    s.hk = w.hk;
    s.t0 = 2 * p.T * w.pair;
    sequence(p, w.b, s.fresh, s.before);
    s.all = pair_tiles(p, s.fresh, s.before, w.pair);
    s.n_all = s.all.count();
    s.j0 = w.j;
    s.n = imin(s.n_all - w.j, w.left);
    const int first = s.before + s.t0, mid = first + p.T, end = s.before + s.fresh;
    s.has_b = mid < end;
    // (tile index to its place in the list)
    const int a_hi = imin(mid, end);  // A's last token + 1
    s.a_end = s.all.lead + ((a_hi - 1) / 128 + 1 - s.all.lo);
    s.b_0 = s.b_1 = 0;
    if (s.has_b) {
        const KeyTiles kb = key_tiles(mid, imin(mid + p.T, end) - 1, p.window, p.sinks);
        s.b_1 = s.all.lead + imax(kb.lo - s.all.lo, 0);
        s.b_0 = kb.lead <= s.all.lead ? kb.lead : s.all.lead + imax(kb.lead - s.all.lo, 0);
    }
    return true;
}
__device__ __forceinline__ void step(const ChunkParams& p, const Segment& s, Walk& w) {
    w.left -= s.n;
    w.j += s.n;
    if (w.left <= 0 || w.j < s.n_all) return;
    w.j = 0;
    ++w.pair;
    int n = s.fresh, before;
    while (w.pair >= pairs_of(p, n)) {  // (the line goes on: some sequence has another pair)
        w.pair = 0;
        if (++w.b == p.B) {
            w.b = 0;
            if (++w.hk == p.Hk) {  // (only if the lengths were changed meanwhile)
                w.left = 0;
                return;
            }
        }
        sequence(p, w.b, n, before);
    }
}

// Tokens lo .. hi - 1 and those below `lead` are seen by some row of the segment's pair.
struct Live {
    int lo, hi, lead;
    __device__ __forceinline__ bool token(int t) const { return t < hi && (t >= lo || t < lead); }
    __device__ __forceinline__ bool any(int t, int n) const { return t < hi && (t + n > lo || t < lead); }
    __device__ __forceinline__ bool every(int t, int n) const { return t + n <= hi && (t >= lo || t + n <= lead); }
};
__device__ __forceinline__ Live live_of(const ChunkParams& p, const Segment& s) {
    return {imax(s.before + s.t0 - p.window + 1, 0), s.before + s.fresh, p.sinks};
}

// The CTA that has unit u.
__device__ __forceinline__ int unit_cta(long long units, int grid, long long u) {
    return (int)(((u + 1) * grid - 1) / units);
}

// Joins the n_parts parts of a pair of query tiles, which CTAs owner, owner + 1, ... left: the tiles' T G rows are
// dealt out to the warps, eight at a time.  O = sum w_i O_i / sum w_i, LSE = log sum exp(LSE_i).
template <int D, bool BF16>
__device__ __noinline__ void join_parts(const ChunkParams& p, int b, int hk, int t0, int fresh, int owner, int n_parts,
                                        int warp, int lane) {
    constexpr int kPer = D / 32, kRows = 8;
    const int per_tile = (p.T * p.group + kRows - 1) / kRows * kRows;
    const int rows = t0 + p.T < fresh ? 2 * per_tile : per_tile;
#pragma unroll 1
    for (int at = warp * kRows; at < rows; at += 8 * kRows) {
        // Rows r0 .. of tile my_t; lane 8 q + r: row r0 + r, of which it takes the log-sum-exp of part q of two.
        const int my_t = at >= per_tile, r0 = at + my_t * (kTileRows - per_tile);
        const int my_r = r0 + (lane & (kRows - 1)), my_row = my_r & (kTileRows - 1);
        const int my_head = my_row / p.T, my_i = t0 + my_t * p.T + my_row - my_head * p.T;
        const bool mine = my_head < p.group && my_i < fresh;
        if (!__any_sync(0xffffffffu, mine)) continue;
        auto part_at = [&](int r, int c) {  // row r of the two tiles
            return (2 * (size_t)(owner + c) + (c == 0 ? 1 : 0)) * (2 * kTileRows) + r;
        };
        float top = -INFINITY, sum = 0.0f, x[kRows][kPer];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[r][e] = 0.0f;
#pragma unroll 1
        for (int c0 = 0; c0 < n_parts; c0 += 2) {  // two parts: their loads are in flight together
            const int q = lane >> 3;
            const float y = mine && q < 2 && c0 + q < n_parts ? __ldcg(p.slot_lse + part_at(my_r, c0 + q)) : -INFINITY;
            float v[2][kRows][kPer];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float* src = p.slot_o + part_at(r0, imin(c0 + c, n_parts - 1)) * D + lane * kPer;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    if constexpr (kPer == 4) {
                        const float4 u = __ldcg(reinterpret_cast<const float4*>(src + (size_t)r * D));
                        v[c][r][0] = u.x;
                        v[c][r][1] = u.y;
                        v[c][r][2] = u.z;
                        v[c][r][3] = u.w;
                    } else {
                        const float2 u = __ldcg(reinterpret_cast<const float2*>(src + (size_t)r * D));
                        v[c][r][0] = u.x;
                        v[c][r][1] = u.y;
                    }
                }
            }
            const float other = __shfl_xor_sync(0xffffffffu, y, 8);  // (lanes 0 .. 15 hold the two parts)
            const float next = fmaxf(top, fmaxf(y, other)), base = next == -INFINITY ? 0.0f : next;
            const float f = ex2_approx(top - base);
            const float w = y == -INFINITY ? 0.0f : ex2_approx(y - base);  // (a NaN stays)
            sum = fmaf(sum, f, w + __shfl_xor_sync(0xffffffffu, w, 8));
            top = next;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float fr = __shfl_sync(0xffffffffu, f, r);
#pragma unroll
                for (int e = 0; e < kPer; ++e) x[r][e] *= fr;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float wr = __shfl_sync(0xffffffffu, w, 8 * c + r);
                    if (wr == 0.0f) continue;  // (of a part without a key nothing was written)
#pragma unroll
                    for (int e = 0; e < kPer; ++e) x[r][e] = fmaf(wr, v[c][r][e], x[r][e]);
                }
            }
        }
        const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;  // (in lanes 0 .. 15)
        const size_t my_orow = (size_t)b * p.Hq + hk * p.group + my_head;
        if (mine && lane < kRows)
            p.lse[my_orow * p.L + my_i] = sum != 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
        uint8_t* my_dst = mine ? reinterpret_cast<uint8_t*>(p.o) + row_offset(p.so, (int)my_orow, p.Hq, my_i) : nullptr;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float f = __shfl_sync(0xffffffffu, inv, r);
            uint8_t* dst = reinterpret_cast<uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(my_dst), r));
            if (!dst) continue;
            uint32_t* d = reinterpret_cast<uint32_t*>(dst) + lane * (kPer / 2);
#pragma unroll
            for (int e = 0; e < kPer; e += 2) d[e / 2] = pack2<BF16>(x[r][e] * f, x[r][e + 1] * f);
        }
    }
}

template <int D, bool BF16, bool Q8>
__global__ void __launch_bounds__(ChunkCfg<D, BF16, Q8>::kThreads, 1)
    fa_chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = ChunkCfg<D, BF16, Q8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    __shared__ uint64_t bar_qf, bar_qe, bar_f[C::kSlots], bar_e[C::kSlots];  // slots full / empty
    __shared__ uint64_t bar_sf[2], bar_pf[2], bar_oready[2], bar_fin;
    __shared__ uint64_t bar_segf[C::kSegs], bar_sege[C::kSegs];  // segments there / taken
    __shared__ Segment seg_sh[C::kSegs];
    __shared__ uint64_t bar_part, bar_ticket;  // a part written by all softmax warps; counted
    __shared__ uint64_t bar_rf[Q8 ? 2 * C::kRaw : 1], bar_re[Q8 ? 2 * C::kRaw : 1];  // bytes landed / read
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ int warp_sum[C::kThreads / 32];
    __shared__ Walk start_sh;
    __shared__ long long total_sh;
    __shared__ int ticket_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_v = &abort_flag;

    if (threadIdx.x == 0) {
        if (p.num_pages > 0) tma_prefetch_desc(&p.tm_q);
        if (p.num_pages > 0) {
            tma_prefetch_desc(&p.tm_k);
            tma_prefetch_desc(&p.tm_v);
        }
        abort_flag = 0;
        start_sh.left = 0;
        mbar_init(&bar_qf, 1);
        mbar_init(&bar_qe, 1);
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&bar_f[s], Q8 ? C::kConverters : 1);
            mbar_init(&bar_e[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar_sf[t], 1);
            mbar_init(&bar_pf[t], 128);
            mbar_init(&bar_oready[t], 1);
        }
        for (int s = 0; s < 2 * C::kRaw; ++s) {
            mbar_init(&bar_rf[s], 1);
            mbar_init(&bar_re[s], C::kConverters);
        }
        for (int s = 0; s < C::kSegs; ++s) {
            mbar_init(&bar_segf[s], 1);
            mbar_init(&bar_sege[s], 10);  // V, MMA and softmax warps
        }
        mbar_init(&bar_part, 8);
        mbar_init(&bar_ticket, 1);
        mbar_init(&bar_fin, 1);
        mbar_fence_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&tmem_base_sh, C::kTmemCols);
    // Query rows behind T G are never written: zeros, so that no leftover score makes a row rescale.
    for (int e = (int)threadIdx.x; e < 2 * C::kChunks * (kTileRows - p.T * p.group) * 8; e += C::kThreads) {
        const int box = e / ((kTileRows - p.T * p.group) * 8), at = e - box * (kTileRows - p.T * p.group) * 8;
        sts_u32x4(smem_u32(smem + C::kOffQ + box * kChunkBytes + p.T * p.group * 128 + at * 16),
                  make_uint4(0u, 0u, 0u, 0u));
    }
    fence_proxy_async_smem();
    // ---- the line: every thread sums a run of (sequence, pair) ----
    const int slots = p.B * p.max_pairs;
    const int run = (slots + C::kThreads - 1) / C::kThreads;
    const int i0 = imin((int)threadIdx.x * run, slots), i1 = imin(i0 + run, slots);
    auto walk_run = [&](auto&& f) {  // f(b, pair, key tiles) for the run, until it returns true
        int b = i0 / p.max_pairs, i = i0 - b * p.max_pairs, n = 0, before = 0, pairs = 0;
        for (int at = i0; at < i1; ++at) {
            if (at == i0 || i == 0) {
                if (!sequence(p, b, n, before) && i == 0 && blockIdx.x == 0)
                    atomicCAS(p.status, 0, (int)kDevBadArg);
                pairs = pairs_of(p, n);
            }
            if (i < pairs && f(b, i, pair_tiles(p, n, before, i).count())) return;
            if (++i == p.max_pairs) {
                i = 0;
                ++b;
            }
        }
    };
    int sum = 0;
    walk_run([&](int, int, int k) {
        sum += k;
        return false;
    });
    int scan = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int before_me = scan - sum, per_head = 0;
    for (int i = 0; i < C::kThreads / 32; ++i) {
        if (i < warp) before_me += warp_sum[i];
        per_head += warp_sum[i];
    }
    const long long total = (long long)per_head * p.Hk;
    const int workers = (int)(total < p.grid ? total : p.grid);
    if ((int)blockIdx.x < workers) {
        const long long u0 = total * blockIdx.x / workers, u1 = total * (blockIdx.x + 1) / workers;
        const int hk = (int)(u0 / per_head), rest = (int)(u0 - (long long)hk * per_head);
        if (rest >= before_me && rest < before_me + sum) {
            int at = before_me;
            walk_run([&](int b, int i, int k) {
                if (rest >= at + k) {
                    at += k;
                    return false;
                }
                start_sh = {hk, b, i, rest - at, (int)(u1 - u0)};
                total_sh = total;
                return true;
            });
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    Walk walk = start_sh;
    // (16-bit) The i-th segment of this CTA, for all warps but K's; false behind the last one, and (ok = false)
    // without it.
    auto take = [&](int i, Segment& s, bool& ok) -> bool {
        const int at = i % C::kSegs;
        ok = wait_warp(&bar_segf[at], (uint32_t)(i / C::kSegs) & 1u, abort_v, p.timeout_ns);
        if (!ok) return false;
        s = seg_sh[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_sege[at]);
        return s.n > 0;
    };

    // (A warpgroup sets its registers with one instruction.)
    if (warp >= 8) {
    if constexpr (Q8) regs_lower<C::kRegsOther>();
    if (warp == C::kKWarp || warp == C::kVWarp) {
        // ------------------------------ TMA producers ------------------------------
        // The K warp brings each segment's query pair, and K's pages; the V warp V's.  Lane 8c + i issues page i
        // of chunk c, over e4m3 lane i page i and lane 8 + i its exponents; table entries are fetched one tile ahead.
        const bool is_k = warp == C::kKWarp;
        const CUtensorMap* map = is_k ? &p.tm_k : &p.tm_v;
        const int my_page = lane & (kPagesPerTile - 1), my_chunk = lane / kPagesPerTile;
        constexpr int kIssuers = Q8 ? 2 : C::kChunks;  // groups of eight lanes
        uint64_t* full = Q8 ? bar_rf : bar_f;
        uint64_t* empty = Q8 ? bar_re : bar_e;
        auto slot_of = [&](int i) { return Q8 ? (is_k ? 0 : C::kRaw) + i % C::kRaw : C::slot(i, !is_k); };
        auto use_of = [&](int i) { return Q8 ? i / C::kRaw : C::use(i, !is_k); };
        constexpr int kRing = Q8 ? C::kRaw : C::kStages;
        bool ok = true;
        int issued = 0, n_seg = 0;
        Segment sg;
        // The next segment, K: worked out and left for the others.
        auto leave = [&](int i) -> bool {
            if (!segment_at(p, walk, sg)) sg.n = 0;
            sg.done = start_sh.left - walk.left;
            const int at = i % C::kSegs;
            if (i >= C::kSegs) ok = wait_warp(&bar_sege[at], (uint32_t)(i / C::kSegs - 1) & 1u, abort_v, p.timeout_ns);
            if (!ok) return false;
            if (lane == 0) {
                seg_sh[at] = sg;
                mbar_arrive(&bar_segf[at]);
            }
            __syncwarp();
            return sg.n > 0;
        };
        int i = 0;
        for (; ok && (Q8 ? segment_at(p, walk, sg) : is_k ? leave(i) : take(i, sg, ok));
             Q8 || is_k ? step(p, sg, walk) : void(), ++i) {
            if (is_k) {
                if (n_seg > 0) ok = wait_warp(&bar_qe, (uint32_t)(n_seg - 1) & 1u, abort_v, p.timeout_ns);
                if (!ok) break;
                if (lane == 0) {
                    const int nt = sg.has_b ? 2 : 1;
                    const uint32_t box = (uint32_t)(p.group * p.T) * kChunkElems * 2;
                    mbar_arrive_expect_tx(&bar_qf, (uint32_t)nt * C::kChunks * box);
                    for (int t = 0; t < nt; ++t)
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_4d(smem + C::kOffQ + t * C::kTileBytes + c * kChunkBytes, &p.tm_q, &bar_qf,
                                        c * kChunkElems, sg.t0 + t * p.T, sg.hk * p.group, sg.b);
                }
                __syncwarp();
                ++n_seg;
            }
            const Live live = live_of(p, sg);
            auto entry = [&](int j) {  // this lane's page of tile j, or -1: nothing of it counts
                const int pg = sg.all.tile(j) * kPagesPerTile + my_page;
                if (my_chunk >= kIssuers || !live.any(pg * kPageTokens, kPageTokens)) return -1;
                const int page = p.block_tables[(size_t)sg.b * p.max_pages + pg];
                if (page < 0 || page >= p.num_pages) {
                    atomicCAS(p.status, 0, (int)kDevBadArg);
                    return -1;
                }
                return page;
            };
            int next = entry(sg.j0);
            for (int j = sg.j0; j < sg.j0 + sg.n; ++j, ++issued) {
                const int page = next;
                if (j + 1 < sg.j0 + sg.n) next = entry(j + 1);
                const int st = slot_of(issued), use = use_of(issued);
                if (use > 0) {
                    ok = wait_warp(&empty[st], ((uint32_t)use & 1u) ^ 1u, abort_v, p.timeout_ns);
                    if (!ok) break;
                }
                const size_t ph = page < 0 ? 0 : (size_t)page * p.Hk + sg.hk;
                const int row = page < 0 ? kPageTokens : 0;  // (outside the map: zeros)
                if constexpr (Q8) {
                    uint8_t* ex = smem + C::kOffExp + st * kTileRows + my_page * kPageTokens;
                    const bool mine = my_chunk == 1 && page >= 0;
                    const uint32_t n_ex = __popc(__ballot_sync(0xffffffffu, mine));
                    if (my_chunk == 1 && page < 0) {  // no page: zeros, whose exponents are finite
                        sts_u32x4(smem_u32(ex), make_uint4(0u, 0u, 0u, 0u));
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kRawBytes + n_ex * kPageTokens);
                    __syncwarp();
                    if (my_chunk == 0)
                        tma_load_3d(smem + C::kOffRaw + st * C::kRawBytes + my_page * (kPageTokens * D), map,
                                    &full[st], 0, row, (int)ph);
                    if (mine) bulk_load(ex, (is_k ? p.k_exp : p.v_exp) + ph * kPageTokens, kPageTokens, &full[st]);
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kTileBytes);
                    __syncwarp();
                    if (my_chunk < kIssuers)
                        tma_load_3d(smem + C::kOffKV + st * C::kTileBytes + my_chunk * kChunkBytes +
                                        my_page * (kPageTokens * 128),
                                    map, &full[st], my_chunk * kChunkElems, row, (int)ph);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        // Drain: the newest fill of every slot must have landed before the CTA exits.
        if (is_k && n_seg > 0) wait_bounded(&bar_qf, (uint32_t)(n_seg - 1) & 1u, nullptr, p.timeout_ns);
        for (int g = issued - 1; g >= 0 && g >= issued - kRing; --g)
            wait_bounded(&full[slot_of(g)], (uint32_t)use_of(g) & 1u, nullptr, p.timeout_ns);
    } else if (warp == C::kMmaWarp) {
        // ------------------------------ MMA issuer ------------------------------
        bool ok = true;
        int g = 0, n_seg = 0, ps[2] = {0, 0};
        const uint32_t neg = p.s_negate ? kIdescNegateA : 0u;
        auto wait_tile = [&](int i, int v) -> bool {  // K or V of the i-th tile is there
            const bool r = wait_warp(&bar_f[C::slot(i, v)], (uint32_t)C::use(i, v) & 1u, abort_v, p.timeout_ns);
            tc_fence_after_sync();
            return r;
        };
        Segment sg;
        int i = 0;
        for (; ok && (Q8 ? segment_at(p, walk, sg) : take(i, sg, ok)); Q8 ? step(p, sg, walk) : void(++i)) {
            const Live live = live_of(p, sg);
            const int j1 = sg.j0 + sg.n;
            const int n_of[2] = {sg.count(0), sg.count(1)};
            int done[2] = {0, 0};
            auto issue_s = [&](int t, int gk) {  // S_t = Q_t K^T for ring fill gk
                const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + C::kOffQ + t * C::kTileBytes));
                const uint64_t kd =
                    sdesc_kmajor_sw128(smem_u32(smem + C::kOffKV + C::slot(gk, 0) * C::kTileBytes));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                    mma_ss_w(tmem + C::kTmS + 128 * t, sdesc_advance(qd, off), sdesc_advance(kd, off),
                             C::kIdescS | neg, kk > 0 ? 1u : 0u);
                }
                mma_commit_w(&bar_sf[t]);
            };
            auto issue_pv = [&](int t, int gv) -> bool {  // O_t += P_t V for ring fill gv (landed)
                if (!wait_warp(&bar_pf[t], (uint32_t)ps[t] & 1u, abort_v, p.timeout_ns)) return false;
                tc_fence_after_sync();
                const uint64_t vd = sdesc_mnmajor_sw128(
                    smem_u32(smem + C::kOffKV + C::slot(gv, 1) * C::kTileBytes), kChunkBytes);
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    mma_ts_w(tmem + C::kTmO + D * t, tmem + C::kTmS + 128 * t + kk * 8,
                             sdesc_advance(vd, kk * 2048), C::kIdescO, (done[t] > 0 || kk > 0) ? 1u : 0u);
                ++ps[t];
                if (++done[t] == n_of[t]) mma_commit_w(&bar_oready[t]);  // O_t is final
                return true;
            };
            ok = wait_warp(&bar_qf, (uint32_t)n_seg & 1u, abort_v, p.timeout_ns);
            tc_fence_after_sync();
            ok = ok && wait_tile(g, 0);
            if (!ok) break;
            for (int t = 0; t < 2; ++t)
                if (sg.active(t, sg.j0)) issue_s(t, g);
            if (sg.n == 1) mma_commit_w(&bar_qe);  // every S of the segment issued
            mma_commit_w(&bar_e[C::slot(g, 0)]);
            for (int j = sg.j0; ok && j < j1; ++j) {
                const bool next = j + 1 < j1;
                const int gj = g + (j - sg.j0);
                // (e4m3: K_{j+1}, which may still be on its way, is waited for behind PV_A.)
                if (!wait_tile(gj, 1) || (!Q8 && next && !wait_tile(gj + 1, 0))) {
                    ok = false;
                    break;
                }
                if constexpr (!Q8) {
                    // Slots of a page that were read with it but hold no token that counts: zeros.
                    const int key0 = sg.all.tile(j) * kTileRows;
                    if (!live.every(key0, kTileRows)) {
                        uint8_t* tile = smem + C::kOffKV + C::slot(gj, 1) * C::kTileBytes;
                        for (int r = lane; r < kTileRows; r += 32) {
                            const int token = key0 + r;
                            if (live.token(token) || !live.any(token & ~(kPageTokens - 1), kPageTokens)) continue;
#pragma unroll
                            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
                                for (int u = 0; u < 8; ++u)
                                    sts_u32x4(smem_u32(tile + c * kChunkBytes + r * 128 + u * 16),
                                              make_uint4(0u, 0u, 0u, 0u));
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok) break;
                    if (sg.active(t, j) && !issue_pv(t, gj)) {
                        ok = false;
                        break;
                    }
                    if (Q8 && t == 0 && next && !wait_tile(gj + 1, 0)) {
                        ok = false;
                        break;
                    }
                    if (next && sg.active(t, j + 1)) issue_s(t, gj + 1);
                }
                if (!ok) break;
                if (j + 2 == j1) mma_commit_w(&bar_qe);  // the segment's last S issued
                mma_commit_w(&bar_e[C::slot(gj, 1)]);
                if (next) mma_commit_w(&bar_e[C::slot(gj + 1, 0)]);
            }
            g += sg.n;
            ++n_seg;
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        mma_commit_w(&bar_fin);  // every issued MMA must finish before TMEM is released
        wait_warp(&bar_fin, 0, nullptr, p.timeout_ns);
    } else if (Q8 && warp >= C::kConvWarp) {
        // ------------------------------ converters ------------------------------
        // Each warp takes eight of every 64 rows of a tile.  Lane 8 q + 4 b + i takes 16-byte units i (and 4 + i) of
        // row q ^ 5b of them: the eight lanes of a shared-memory access then read and write all eight 16-byte
        // places of a line of banks.
        if constexpr (Q8) {
            constexpr int kRows = kTileRows / (8 * C::kConverters), kUnits = kRows * C::kChunks;
            const int unit = lane & 3, row_in = (warp - C::kConvWarp) * 8 + ((lane >> 3) ^ (5 * ((lane >> 2) & 1)));
            bool ok = true;
            int g = 0;  // tiles so far
            Segment sg;
            for (; ok && segment_at(p, walk, sg); step(p, sg, walk)) {
                const Live live = live_of(p, sg);
                for (int j = sg.j0; ok && j < sg.j0 + sg.n; ++j, ++g) {
                    const int key0 = sg.all.tile(j) * kTileRows;
                    // One copy of the code for K and V: with two (and more of it unrolled) the warps of an SM no
                    // longer found their instructions in its cache (2.5 of 10.7 cycles per instruction; 0.5 in
                    // the kernel of 16-bit caches).
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        const int slot = C::slot(g, v), use = C::use(g, v), st = v * C::kRaw + g % C::kRaw;
                        ok = wait_warp(&bar_rf[st], (uint32_t)(g / C::kRaw) & 1u, abort_v, p.timeout_ns);
                        if (!ok) break;
                        const uint32_t raw = smem_u32(smem + C::kOffRaw + st * C::kRawBytes);
                        const uint8_t* ex = smem + C::kOffExp + st * kTileRows;
                        const uint32_t tile = smem_u32(smem + C::kOffKV + slot * C::kTileBytes);
                        uint4 x[kUnits];  // (all reads first: they and the writes keep their order)
                        float f[kRows];
                        auto row_of = [&](int k) { return row_in + 8 * C::kConverters * k; };
#pragma unroll
                        for (int k = 0; k < kRows; ++k) {
                            const int r = row_of(k);
#pragma unroll
                            for (int c = 0; c < C::kChunks; ++c)
                                x[k * C::kChunks + c] =
                                    lds_u32x4(D == 128 ? raw + r * 128 + (uint32_t)((c * 4 + unit) ^ (r & 7)) * 16
                                                       : raw + r * 64 + (uint32_t)(unit ^ ((r >> 1) & 3)) * 16);
                            f[k] = row_scale(ex[r]);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar_re[st]);
                        if (!live.every(key0, kTileRows)) {  // tokens that nobody sees: zeros
#pragma unroll
                            for (int k = 0; k < kRows; ++k) {
                                if (live.token(key0 + row_of(k))) continue;
                                f[k] = 0.0f;
#pragma unroll
                                for (int c = 0; c < C::kChunks; ++c)
                                    x[k * C::kChunks + c] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                        if (use > 0) ok = wait_warp(&bar_e[slot], ((uint32_t)use & 1u) ^ 1u, abort_v, p.timeout_ns);
                        if (!ok) break;
#pragma unroll
                        for (int k = 0; k < kRows; ++k) {
                            const int row = row_of(k);
#pragma unroll
                            for (int c = 0; c < C::kChunks; ++c) {
                                uint32_t y[8];
                                scaled16<BF16>(x[k * C::kChunks + c], f2_make(f[k], f[k]), y);
                                const uint32_t line = tile + c * kChunkBytes + row * 128;
                                sts_u32x4(line + ((uint32_t)((2 * unit) ^ (row & 7)) << 4),
                                          make_uint4(y[0], y[1], y[2], y[3]));
                                sts_u32x4(line + ((uint32_t)((2 * unit + 1) ^ (row & 7)) << 4),
                                          make_uint4(y[4], y[5], y[6], y[7]));
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar_f[slot]);
                    }
                }
            }
            if (!ok && lane == 0) record_timeout(p.status, abort_v);
        }
    }
    } else {
        // ------------------------------ softmax warps ------------------------------
        if constexpr (Q8) regs_raise<C::kRegsSoftmax>();
        // While the first tiles are on their way: the rows without a token get zeros and -inf, 64 rows of a head
        // at a time.
        const int blocks_l = (p.L + 63) / 64;
        const long long fills = (long long)p.B * p.Hq * blocks_l;
        for (long long it = (long long)blockIdx.x * 8 + warp; it < fills; it += (long long)gridDim.x * 8) {
            const int bh = (int)(it / blocks_l), i0 = (int)(it - (long long)bh * blocks_l) * 64;
            int n, ahead;
            sequence(p, bh / p.Hq, n, ahead);
            const int from = imax(n, i0), to = imin(i0 + 64, p.L);
            for (int e = lane; e < (to - from) * (D / 8); e += 32) {
                const int i = from + e / (D / 8), u = e % (D / 8);
                reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.o) + row_offset(p.so, bh, p.Hq, i))[u] =
                    make_uint4(0u, 0u, 0u, 0u);
                if (u == 0) p.lse[(size_t)bh * p.L + i] = -INFINITY;
            }
        }
        const int t = warp / 4, quad = warp % 4;
        const int row = quad * 32 + lane;  // row inside the tile == TMEM lane
        const int head = row / p.T, tok = row - head * p.T;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + C::kTmS + 128 * t;
        const uint32_t o_addr = tmem + lane_off + C::kTmO + D * t;
        const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
        bool ok = true;
        int ps = 0, n_done = 0, n_cut = 0;
        Segment sg;
        int i = 0;
        for (; ok && (Q8 ? segment_at(p, walk, sg) : take(i, sg, ok)); Q8 ? step(p, sg, walk) : void(++i)) {
            const int j1 = sg.j0 + sg.n, cnt = sg.count(t);
            const int first = sg.before + sg.t0 + t * p.T, pos = first + tok;
            const int last = imin(first + p.T, sg.before + sg.fresh) - 1;
            float m_ref = -INFINITY, l_sum = 0.0f;
            bool began = false;
            for (int j = sg.j0; j < j1; ++j) {
                if (!sg.active(t, j)) continue;
                ok = wait_warp(&bar_sf[t], (uint32_t)ps & 1u, abort_v, p.timeout_ns);
                if (!ok) break;
                ++ps;
                tc_fence_after_sync();
                float s[128];
                {
                    uint32_t r[128];
                    tmem_ld_cols<128>(s_addr, r);
#pragma unroll
                    for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(r[i]);
                }
                const int key0 = sg.all.tile(j) * kTileRows;
                if (hides_later(key0, kTileRows, first)) {
                    const int lim = pos - key0;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > lim) s[c] = -INFINITY;
                }
                if (hides_earlier(key0, kTileRows, last, p.window, p.sinks)) {
                    const int lim = pos - p.window - key0, sink = p.sinks - key0;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c <= lim && c >= sink) s[c] = -INFINITY;
                }
                float m4[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) m4[v] = fmaxf(s[v], s[v + 4]);
#pragma unroll
                for (int c = 8; c < 128; c += 8) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) m4[v] = fmax3(m4[v], s[c + v], s[c + 4 + v]);
                }
                const float m_cand = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * p.scale_log2;
                float m_new = m_ref;
                if (m_cand > m_ref + (kRescaleThreshold + kLift<BF16>)) m_new = m_cand - kLift<BF16>;
                const bool rescale = began && (m_new != m_ref);
                const float m_use = (m_new == -INFINITY) ? 0.0f : m_new;
                const float alpha = rescale ? ex2_approx(m_ref - m_new) : 1.0f;
                const uint64_t shift2 = f2_make(-m_use, -m_use);
                uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float y0, y1;
                        f2_split(f2_fma(f2_make(s[h * 32 + 2 * i], s[h * 32 + 2 * i + 1]), scale2, shift2),
                                 y0, y1);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        sum2[i & 1] = f2_add(sum2[i & 1], f2_make(p0, p1));
                        pk[i] = pack2<BF16>(p0, p1);
                    }
                    tmem_st16(s_addr + h * 16, pk);
                }
                float sa, sb, sc, sd;
                f2_split(sum2[0], sa, sb);
                f2_split(sum2[1], sc, sd);
                l_sum = l_sum * alpha + ((sa + sb) + (sc + sd));
                if (__any_sync(0xffffffffu, rescale)) tmem_row_scale<D>(o_addr, alpha);
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(&bar_pf[t]);
                m_ref = m_new;
                began = true;
            }
            if (!ok) break;
            const bool valid = head < p.group && sg.t0 + t * p.T + tok < sg.fresh;
            const bool whole = sg.whole(), behind = !whole && sg.j0 == 0;  // (behind: it goes on in the next CTA)
            const size_t slot = 2 * (size_t)blockIdx.x + (behind ? 1 : 0);
            const size_t part = (slot * 2 + t) * kTileRows + row;
            if (cnt > 0) {
                ok = wait_warp(&bar_oready[t], (uint32_t)n_done & 1u, abort_v, p.timeout_ns);
                if (!ok) break;
                tc_fence_after_sync();
                ++n_done;
            }
            const float lse2 = l_sum != 0.0f ? m_ref + log2f(l_sum) : -INFINITY;
            const float inv_l = l_sum != 0.0f ? 1.0f / l_sum : 0.0f;
            if (whole) {
                const int h = sg.hk * p.group + head;
                const size_t orow = (size_t)sg.b * p.Hq + h;
                const int new_i = sg.t0 + t * p.T + tok;
                if (valid) p.lse[orow * p.L + new_i] = lse2 * kLn2;
                uint8_t* dst = valid ? reinterpret_cast<uint8_t*>(p.o) +
                                           row_offset(p.so, (int)orow, p.Hq, new_i)
                                     : nullptr;
                if (cnt > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t m[8][4];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t r[32];
                            tmem_ld32(o_addr + 64 * c + 32 * hf, r);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                m[4 * hf + e / 4][e % 4] = pack2<BF16>(__uint_as_float(r[2 * e]) * inv_l,
                                                                       __uint_as_float(r[2 * e + 1]) * inv_l);
                        }
                        rows_out(m, dst ? dst + c * 128 : nullptr, lane);
                    }
                }
            } else {
                if (valid) p.slot_lse[part] = cnt > 0 ? lse2 : -INFINITY;
                if (cnt > 0) {
                    float* dst = valid ? p.slot_o + part * D : nullptr;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t r[32], m[8][4];
                        tmem_ld32(o_addr + 32 * c, r);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            m[e / 4][e % 4] = __float_as_uint(__uint_as_float(r[e]) * inv_l);
                        rows_out(m, dst ? reinterpret_cast<uint8_t*>(dst + c * 32) : nullptr, lane);
                    }
                }
                // The CTA that ends the pair's last part joins them all.
                const long long x0 = total_sh * blockIdx.x / workers + (Q8 ? start_sh.left - walk.left : sg.done) - sg.j0;
                const int owner = unit_cta(total_sh, workers, x0);
                const int n_parts = unit_cta(total_sh, workers, x0 + sg.n_all - 1) - owner + 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_part);
                if (warp == 0) {
                    ok = wait_warp(&bar_part, (uint32_t)n_cut & 1u, abort_v, p.timeout_ns);
                    if (!ok) break;
                    if (lane == 0) {
                        pdl_wait();  // the counters are zeroed
                        // The thread that counts fences on both sides: its atomic alone orders nothing, and the
                        // barriers carry the other warps' stores to it, and what it has seen to their loads.
                        __threadfence();
                        *reinterpret_cast<volatile int*>(&ticket_sh) = atomicAdd(&p.counters[owner], 1);
                        __threadfence();
                        mbar_arrive(&bar_ticket);
                    }
                    __syncwarp();
                }
                ok = wait_warp(&bar_ticket, (uint32_t)n_cut & 1u, abort_v, p.timeout_ns);
                if (!ok) break;
                ++n_cut;
                if (*reinterpret_cast<volatile int*>(&ticket_sh) == n_parts - 1)
                    join_parts<D, BF16>(p, sg.b, sg.hk, sg.t0, sg.fresh, owner, n_parts, warp, lane);
            }
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
    }

    if (blockIdx.x == 0) pdl_wait();  // the kernel in front has ended before this one does
    tc_fence_before_sync();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// The counters of the pairs that are cut.
__global__ void __launch_bounds__(kChunkGrid) fa_chunk_zero_kernel(int* counters, int n) {
    pdl_launch_dependents();
    if ((int)threadIdx.x < n) counters[threadIdx.x] = 0;
}

template <int D, bool BF16, bool Q8>
cudaError_t launch_t(const ChunkParams& p, cudaStream_t s) {
    using C = ChunkCfg<D, BF16, Q8>;
    constexpr auto kern = fa_chunk_kernel<D, BF16, Q8>;
    const cudaError_t e = allow_shared_once<kern>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_kernel_early(kern, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmemBytes, s, p);
}

}  // namespace

void chunk_plan(int B, int Hk, int group, int L, int max_pages, ChunkParams* p) {
    p->T = imin(kTileRows / group, imax(L, 1));
    p->max_pairs = (L + 2 * p->T - 1) / (2 * p->T);
    const long long units = (long long)B * Hk * p->max_pairs * ((max_pages + kPagesPerTile - 1) / kPagesPerTile);
    p->grid = (int)(units < 1 ? 1 : units < kChunkGrid ? units : kChunkGrid);
}

cudaError_t launch_chunk(const ChunkParams& p, int D, bool bf16, bool q8, cudaStream_t s) {
    if (D == 64) {
        if (q8) return bf16 ? launch_t<64, true, true>(p, s) : launch_t<64, false, true>(p, s);
        return bf16 ? launch_t<64, true, false>(p, s) : launch_t<64, false, false>(p, s);
    }
    if (q8) return bf16 ? launch_t<128, true, true>(p, s) : launch_t<128, false, true>(p, s);
    return bf16 ? launch_t<128, true, false>(p, s) : launch_t<128, false, false>(p, s);
}

cudaError_t launch_chunk_zero(const ChunkParams& p, cudaStream_t s) {
    return launch_kernel(fa_chunk_zero_kernel, dim3(1), dim3(kChunkGrid), 0, s, p.counters, p.grid);
}

}  // namespace fa
