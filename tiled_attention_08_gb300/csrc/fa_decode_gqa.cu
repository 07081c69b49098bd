// fa_decode_gqa.cu -- one decode step with grouped heads over a 16-bit or e4m3 paged cache (sm_103a).
//
// Query rows q[b, h], h = hk * G .. hk * G + G - 1, share the cache head hk:
//     O[b,h] = softmax(scale * q[b,h] K^T) V,  LSE[b,h] = log sum exp(scale * q[b,h] . k_t),
// over the seq_lens[b] tokens of the sequence, token t in page block_tables[b][t / 16] at slot
// t % 16.  A cached e4m3 row is its values times a power of two (fa_e4m3.cuh).
//
// Bound by HBM: every cached row is read once per cache head and used by G query rows, 4 G D FLOPs
// for 2 D or 4 D bytes.  On the FMA pipes the products alone would cost G instructions per value
// and lane, over the issue rate from G = 4 on, so they run on the tensor cores.  tcgen05's
// smallest tile has 64 rows and reads its operands from shared memory, where e4m3 rows would
// first have to be written back as 16-bit; mma.sync m16n8k16 takes its operands from registers,
// where the conversion costs one instruction per two values, and its 8 columns are the group.
// The keys are its 16 rows: S^T = K Q^T (16 keys = one page, 8 queries) and O^T += V^T P^T.  At
// the rate HBM delivers the tensor pipe is under a fifth busy.
//
// A CTA is one (sequence, cache head, block of 8 or 16 queries, split of the pages); its four warps
// take pages in turn, each with its own ring of page slots filled by TMA (one lane issues, an
// mbarrier per slot), so that no warp waits for another before the end.  Operand layouts, with
// lane = 4 g + t as the mma defines them:
//  * K, A operand (rows g, g+8 = keys): the contraction runs over D in any order that Q follows,
//    so a lane reads whole 16-byte units of its two rows, units 2t and 2t+1 of each 128-byte row;
//  * S^T comes out with its columns (queries 2t, 2t+1) in the lane that also holds O^T's columns,
//    so each lane keeps the running statistics of its own two queries;
//  * P^T, B operand: S^T's 8 x 8 blocks transposed in registers (movmatrix);
//  * V^T, A operand (rows = elements, contraction over keys 2t, 2t+1, 2t+8, 2t+9): a lane reads unit
//    g of its four keys; bytes (or halves) of two keys are paired by byte permutes.
// The TMA's 128-byte (64-byte) swizzle spreads these reads over all banks.
//
// Softmax in the log2 domain.  The reference of a column is only raised when a score exceeds it
// by more than 2^8 (a warp vote), so the maximum over the lanes is rarely taken.  An e4m3 cache
// needs two references: the sum of weights takes p_j = 2^(y_j - m); the products take
// a_j = 2^(y_j + ev_j - mo) with the value row's exponent ev_j, so that a weight times its row's
// scale neither overflows nor is lost in fp16, whatever the rows' magnitudes.  P is rounded to the
// cache's 16-bit type (fp16 for e4m3: 2^-12), as in the prefill kernels; sums stay fp32.
#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;  // log2 headroom of the references
constexpr int kWarps = 4;

// Q8: an e4m3 cache.
template <int D, bool Q8>
struct GqaCfg {
    static constexpr int kRowBytes = (D * (Q8 ? 1 : 2)) < 128 ? 64 : 128;  // of one TMA box
    static constexpr int kBoxes = D * (Q8 ? 1 : 2) / kRowBytes;
    static constexpr int kBoxBytes = kPageTokens * kRowBytes;
    static constexpr int kPageBytes = kBoxes * kBoxBytes;
    static constexpr int kSteps = D / 16;   // contraction steps of S^T
    static constexpr int kTiles = D / 16;   // 16-element row tiles of O^T
    // Page slots per warp: about 48-64 KB per CTA.
    static constexpr int kStages = Q8 ? (D == 128 ? 4 : 6) : (D == 128 ? 3 : 4);
    static int smem_bytes(int stages) {
        return kWarps * stages * (2 * kPageBytes + (Q8 ? 32 : 0)) + 1024;
    }
};

__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                              int page_head) {
    tma_load_3d(dst, map, bar, x, 0, page_head);
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Maximum over the lanes that hold the same column (lanes with the same t).
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// Raises a reference to the column's maximum; returns the factor of what was summed under it.
__device__ __forceinline__ float raise(float& ref, float top) {
    const float next = fmaxf(ref, column_max(top));
    const float f = next == -INFINITY ? 1.0f : ex2_approx(ref - next);
    ref = next;
    return f;
}

// BF16: the type of q and o (and of a 16-bit cache).  NT: blocks of 8 queries.
template <int D, bool Q8, bool BF16, int NT>
__global__ void __launch_bounds__(kWarps * 32)
    fa_decode_gqa_kernel(const __grid_constant__ GqaParams p) {
    using C = GqaCfg<D, Q8>;
    constexpr bool kMmaBf16 = BF16 && !Q8;  // e4m3 values are exact in fp16
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    __shared__ uint64_t bar_full[kWarps][16];
    __shared__ float red_m[kWarps][NT * 8], red_mo[kWarps][NT * 8], red_l[kWarps][NT * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x, b = blockIdx.z;
    const int hk = (int)blockIdx.y / p.q_blocks, qb = (int)blockIdx.y - hk * p.q_blocks;
    const int q0 = qb * (NT * 8);                    // first query of this block in the group
    const int n_q = min(NT * 8, p.group - q0);       // queries of this block
    const size_t row0 = (size_t)b * p.Hq + (size_t)hk * p.group + q0;
    const int stages = p.stages;

    pdl_launch_dependents();
    int n = p.seq_lens[b];
    if (n < 0 || n > (long long)p.max_pages * kPageTokens || (n > 0 && p.num_pages == 0)) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, (int)kDevBadArg);
        n = 0;
    }
    const int n_pages = (n + kPageTokens - 1) / kPageTokens;
    const int pg0 = split * p.pages_per_split;
    const int pg1 = min(n_pages, pg0 + p.pages_per_split);
    if (pg0 >= pg1) {  // no key in this split
        if (threadIdx.x < n_q) {
            if (p.part_o)
                p.part_lse[(row0 + threadIdx.x) * p.parts + p.part0 + split] = -INFINITY;
            else
                p.lse[row0 + threadIdx.x] = -INFINITY;
        }
        if (!p.part_o)
            for (int i = threadIdx.x; i < n_q * D / 2; i += kWarps * 32)
                reinterpret_cast<uint32_t*>(p.o)[row0 * D / 2 + i] = 0u;
        pdl_wait();
        return;
    }

    if (lane < stages) mbar_init(&bar_full[warp][lane], 1);
    mbar_fence_init();
    __syncwarp();

    // This warp's pages: pg0 + warp, + 4, ...; the ring runs `stages` pages ahead.
    const int mine = (pg1 - pg0 - warp + kWarps - 1) / kWarps;  // pages of this warp (may be 0)
    uint8_t* ring = smem + (size_t)warp * stages * (2 * C::kPageBytes);
    uint8_t* exps = smem + (size_t)kWarps * stages * (2 * C::kPageBytes) + warp * stages * 32;
    const int* table = p.block_tables + (size_t)b * p.max_pages + pg0 + warp;
    auto entry = [&](int i) { return i < mine ? table[(size_t)i * kWarps] : 0; };
    int cur = entry(lane), nxt = entry(32 + lane);  // table entries of the next 32 + 32 pages
    auto issue = [&](int i) {  // page i of this warp into slot i % stages; the whole warp calls it
        if (i > 0 && (i & 31) == 0) {
            cur = nxt;
            nxt = entry(i + 32 + lane);
        }
        int phys = __shfl_sync(0xffffffffu, cur, i & 31);
        if (lane == 0) {
            const bool bad = phys < 0 || phys >= p.num_pages;
            if (bad) {  // report it and read page 0 instead: nothing outside the cache is touched
                atomicCAS(p.status, 0, (int)kDevBadArg);
                phys = 0;
            }
            const int st = i % stages;
            uint64_t* bar = &bar_full[warp][st];
            uint8_t* dst = ring + st * (2 * C::kPageBytes);
            const int ph = phys * p.Hk + hk;
            mbar_arrive_expect_tx(bar, 2 * C::kPageBytes + (Q8 ? 32 : 0));
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
                tma_load_page(dst + x * C::kBoxBytes, &p.tm_k, bar, x * 64, ph);
            if constexpr (Q8) {
                bulk_load(exps + st * 32, p.k_exp + (size_t)ph * kPageTokens, 16, bar);
                bulk_load(exps + st * 32 + 16, p.v_exp + (size_t)ph * kPageTokens, 16, bar);
            }
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
                tma_load_page(dst + C::kPageBytes + x * C::kBoxBytes, &p.tm_v, bar, x * 64, ph);
        }
    };
    const int ahead = min(stages, mine);
    for (int i = 0; i < ahead; ++i) issue(i);

    // Q fragments (B operand).  Step s of lane t covers elements elem(s) .. + 3: the order in
    // which the K rows are read below.
    uint32_t qf[C::kSteps][NT][2];
    float q_factor[NT][2];  // factor of S^T's columns 2t, 2t+1: scale * log2(e), and for e4m3 the
                            // power of two that brought the query row into fp16's range
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int qi = nt * 8 + g;
        const uint8_t* src = static_cast<const uint8_t*>(p.q) + (row0 + qi) * D * 2;
        uint32_t w[C::kSteps][2];
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
            const int e = Q8 ? (D / 4) * t + 4 * s : 64 * (s >> 2) + 16 * t + 4 * (s & 3);
            uint2 u = make_uint2(0u, 0u);
            if (qi < n_q) u = *reinterpret_cast<const uint2*>(src + e * 2);
            w[s][0] = u.x;
            w[s][1] = u.y;
        }
        float f = 1.0f;  // the row's power of two
        if constexpr (Q8 && BF16) {
            uint32_t mx = 0;
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    mx = max(mx, max((w[s][j] << 16) & 0x7fff0000u, w[s][j] & 0x7fff0000u));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // Largest magnitude to [2^14, 2^15); 2^100 at most (rows below 2^-86 lose nothing
            // that a score could show).
            const int ex = (int)(mx >> 23) - 127;
            if (mx != 0 && mx < 0x7f800000u) f = __uint_as_float((uint32_t)(127 + min(14 - ex, 100)) << 23);
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 v = unpack2<true>(w[s][j]);
                    w[s][j] = pack2<false>(v.x * f, v.y * f);
                }
        }
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
            qf[s][nt][0] = w[s][0];
            qf[s][nt][1] = w[s][1];
        }
        const float back = p.scale_log2 / f;
        q_factor[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);      // lane of g = 2t
        q_factor[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);  // lane of g = 2t + 1
    }

    float acc[C::kTiles][NT][4];
    float m[NT][2], mo[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[nt][j] = mo[nt][j] = -INFINITY;
            l[nt][j] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][nt][j] = 0.0f;
    }

    bool ok = true;
    int done = 0;
    for (; done < mine; ++done) {
        const int st = done % stages;
        ok = wait_warp(&bar_full[warp][st], (uint32_t)(done / stages) & 1u, nullptr, p.timeout_ns);
        if (!ok) break;
        const uint8_t* kp = ring + st * (2 * C::kPageBytes);
        const uint8_t* vp = kp + C::kPageBytes;
        const uint32_t ks = smem_u32(kp), vs = smem_u32(vp);
        float c[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[nt][j] = 0.0f;
        // ---- S^T = K Q^T: rows g and g + 8 of the page ----
        if constexpr (!Q8) {
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t u = (uint32_t)((2 * t + hf) ^ g) * 16;
                    const uint4 lo = lds_u32x4(ks + x * C::kBoxBytes + g * 128 + u);
                    const uint4 hi = lds_u32x4(ks + x * C::kBoxBytes + (g + 8) * 128 + u);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int s = 4 * x + 2 * hf;
                        mma16816<kMmaBf16>(c[nt], lo.x, hi.x, lo.y, hi.y, qf[s][nt][0], qf[s][nt][1]);
                        mma16816<kMmaBf16>(c[nt], lo.z, hi.z, lo.w, hi.w, qf[s + 1][nt][0],
                                           qf[s + 1][nt][1]);
                    }
                }
            }
        } else {
            constexpr int kUnits = D / 64;  // 16-byte units of a row per lane
#pragma unroll
            for (int hf = 0; hf < kUnits; ++hf) {
                uint32_t alo, ahi;
                if constexpr (D == 128) {
                    const uint32_t u = (uint32_t)((2 * t + hf) ^ g) * 16;
                    alo = ks + g * 128 + u;
                    ahi = ks + (g + 8) * 128 + u;
                } else {  // 64-byte rows: unit index XOR (row / 2) % 4
                    alo = ks + g * 64 + (uint32_t)(t ^ ((g >> 1) & 3)) * 16;
                    ahi = alo + 8 * 64;
                }
                const uint4 lo = lds_u32x4(alo), hi = lds_u32x4(ahi);
                const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = e4m3x2_to_f16x2(wl[i] & 0xffffu), a2 = e4m3x2_to_f16x2(wl[i] >> 16);
                    const uint32_t a1 = e4m3x2_to_f16x2(wh[i] & 0xffffu), a3 = e4m3x2_to_f16x2(wh[i] >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<false>(c[nt], a0, a1, a2, a3, qf[4 * hf + i][nt][0], qf[4 * hf + i][nt][1]);
                }
            }
        }
        // ---- online softmax over the page ----
        const int left = n - (pg0 + warp + done * kWarps) * kPageTokens;  // tokens from this page on
        const bool partial = left < kPageTokens;
        float fk[2] = {1.0f, 1.0f}, ev[2] = {0.0f, 0.0f};  // rows g, g + 8
        if constexpr (Q8) {
            const uint8_t* ex = exps + st * 32;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                fk[r] = row_scale(ex[g + 8 * r]);
                const uint32_t E = ex[16 + g + 8 * r];
                ev[r] = E == kExpNan ? __uint_as_float(0x7fc00000u) : (float)((int)E - 127);
            }
        }
        float z[NT][4];
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j >> 1;
                float y = c[nt][j] * q_factor[nt][j & 1];
                if constexpr (Q8) y *= fk[r];
                float zz = Q8 ? y + ev[r] : y;
                if (partial && g + 8 * r >= left) y = zz = -INFINITY;
                c[nt][j] = y;
                z[nt][j] = zz;
                up |= y > m[nt][j & 1] + kRaise;
                if constexpr (Q8) up |= zz > mo[nt][j & 1] + kRaise;
            }
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float f = raise(m[nt][j], fmaxf(c[nt][j], c[nt][j + 2]));
                    l[nt][j] *= f;
                    const float fo = Q8 ? raise(mo[nt][j], fmaxf(z[nt][j], z[nt][j + 2])) : f;
#pragma unroll
                    for (int i = 0; i < C::kTiles; ++i) {
                        acc[i][nt][j] *= fo;
                        acc[i][nt][j + 2] *= fo;
                    }
                }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float a[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ref = m[nt][j & 1];
                const float pj = ex2_approx(c[nt][j] - (ref == -INFINITY ? 0.0f : ref));
                l[nt][j & 1] += pj;
                a[j] = pj;
                if constexpr (Q8) {
                    const float ro = mo[nt][j & 1];
                    a[j] = ex2_approx(z[nt][j] - (ro == -INFINITY ? 0.0f : ro));
                }
            }
            pf[nt][0] = transpose8x8(pack2<kMmaBf16>(a[0], a[1]));
            pf[nt][1] = transpose8x8(pack2<kMmaBf16>(a[2], a[3]));
        }
        // ---- O^T += V^T P^T: keys 2t, 2t+1, 2t+8, 2t+9 of the page ----
        // Slots past the sequence's end hold anything: their values count as zeros (their weights
        // are zero, but zero times a NaN is not).
        const bool dead[4] = {partial && 2 * t >= left, partial && 2 * t + 1 >= left,
                              partial && 2 * t + 8 >= left, partial && 2 * t + 9 >= left};
        if constexpr (!Q8 || D == 128) {
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = 2 * t + (k & 1) + 8 * (k >> 1);
                    v[k] = lds_u32x4(vs + x * C::kBoxBytes + key * 128 + (uint32_t)(g ^ (key & 7)) * 16);
                    if (dead[k]) v[k] = make_uint4(0u, 0u, 0u, 0u);
                }
                const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w},
                                          {v[1].x, v[1].y, v[1].z, v[1].w},
                                          {v[2].x, v[2].y, v[2].z, v[2].w},
                                          {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (!Q8) {
                        const uint32_t a0 = __byte_perm(w[0][i], w[1][i], 0x5410);
                        const uint32_t a1 = __byte_perm(w[0][i], w[1][i], 0x7632);
                        const uint32_t a2 = __byte_perm(w[2][i], w[3][i], 0x5410);
                        const uint32_t a3 = __byte_perm(w[2][i], w[3][i], 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<kMmaBf16>(acc[4 * x + i][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                    } else {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t lo = __byte_perm(w[0][i], w[1][i], hf ? 0x7362 : 0x5140);
                            const uint32_t hi = __byte_perm(w[2][i], w[3][i], hf ? 0x7362 : 0x5140);
                            const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xffffu), a1 = e4m3x2_to_f16x2(lo >> 16);
                            const uint32_t a2 = e4m3x2_to_f16x2(hi & 0xffffu), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(acc[2 * i + hf][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                        }
                    }
                }
            }
        } else {  // e4m3, 64-byte rows: 8 elements per lane and key
            uint2 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = 2 * t + (k & 1) + 8 * (k >> 1);
                const uint32_t at = vs + key * 64 + (uint32_t)((g >> 1) ^ ((key >> 1) & 3)) * 16 + (g & 1) * 8;
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[k].x), "=r"(v[k].y) : "r"(at) : "memory");
                if (dead[k]) v[k] = make_uint2(0u, 0u);
            }
            const uint32_t w[4][2] = {{v[0].x, v[0].y}, {v[1].x, v[1].y}, {v[2].x, v[2].y}, {v[3].x, v[3].y}};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t lo = __byte_perm(w[0][i], w[1][i], hf ? 0x7362 : 0x5140);
                    const uint32_t hi = __byte_perm(w[2][i], w[3][i], hf ? 0x7362 : 0x5140);
                    const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xffffu), a1 = e4m3x2_to_f16x2(lo >> 16);
                    const uint32_t a2 = e4m3x2_to_f16x2(hi & 0xffffu), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<false>(acc[2 * i + hf][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            }
        }
        __syncwarp();  // every lane has read the slot
        if (done + stages < mine) issue(done + stages);
    }
    if (!ok) {
        if (lane == 0) atomicCAS(p.status, 0, (int)kDevTimeout);
        // No copy may still be landing when the CTA exits.
        for (int i = done; i < min(mine, done + stages); ++i)
            wait_bounded(&bar_full[warp][i % stages], (uint32_t)(i / stages) & 1u, nullptr, p.timeout_ns);
    }

    // ---- merge the four warps ----
    // Lane (g, t) holds, for queries 2t and 2t+1, the elements e0 + 2i, e0 + 2i + 1 of tile i.
    __syncthreads();  // every warp is done with its ring
    float* red_o = reinterpret_cast<float*>(smem);  // [warp][query][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float sum = column_sum(l[nt][j]);
            const int qi = nt * 8 + 2 * t + j;
            if (g == 0) {
                red_m[warp][qi] = m[nt][j];
                red_mo[warp][qi] = Q8 ? mo[nt][j] : m[nt][j];
                red_l[warp][qi] = sum;
            }
            if (qi < n_q) {
                float* dst = red_o + ((size_t)warp * (NT * 8) + qi) * D;
#pragma unroll
                for (int i = 0; i < C::kTiles; ++i) {
                    const int e = Q8 ? (D / 8) * g + 2 * i : 64 * (i >> 2) + 8 * g + 2 * (i & 3);
                    *reinterpret_cast<float2*>(dst + e) = make_float2(acc[i][nt][j], acc[i][nt][j + 2]);
                }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_q * (D / 2); i += kWarps * 32) {
        const int qi = i / (D / 2), e = (i - qi * (D / 2)) * 2;
        float M = -INFINITY, MO = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            M = fmaxf(M, red_m[w][qi]);
            MO = fmaxf(MO, red_mo[w][qi]);
        }
        float L = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // A warp without pages (or whose scores are all -inf) has references of -inf.
            const float fl = red_m[w][qi] == -INFINITY ? (M == -INFINITY ? 1.0f : 0.0f) : ex2_approx(red_m[w][qi] - M);
            const float fo = red_mo[w][qi] == -INFINITY ? (MO == -INFINITY ? 1.0f : 0.0f) : ex2_approx(red_mo[w][qi] - MO);
            const float2 v = *reinterpret_cast<const float2*>(red_o + ((size_t)w * (NT * 8) + qi) * D + e);
            L = fmaf(red_l[w][qi], fl, L);
            x = fmaf(v.x, fo, x);
            y = fmaf(v.y, fo, y);
        }
        // The two references' distance in two steps: 2^(MO - M) alone may be below fp32's range.
        // (L = 0: every score is -inf, as if the row saw no key.)
        const float f = L == 0.0f ? 0.0f : 1.0f / L;
        const float hop = (!Q8 || MO == -INFINITY || M == -INFINITY) ? 1.0f : ex2_approx(0.5f * (MO - M));
        x = x * f * hop * hop;
        y = y * f * hop * hop;
        const float lse2 = M + log2f(L);
        const size_t row = row0 + qi;
        if (p.part_o) {
            const size_t part = row * p.parts + p.part0 + split;
            *reinterpret_cast<float2*>(p.part_o + part * D + e) = make_float2(x, y);
            if (e == 0) p.part_lse[part] = lse2;
        } else {
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * D + e) = pack2<BF16>(x, y);
            if (e == 0) p.lse[row] = lse2 * kLn2;
        }
    }
    // Launched early behind a kernel that writes other parts of the same rows, this kernel ends
    // only after that one, so that the merge waits for both by waiting for this one.
    pdl_wait();
}

// Merges the parts of each query row: O = sum w_i O_i / sum w_i, LSE = log sum exp(LSE_i), with
// w_i = 2^(LSE2_i - max).  One warp per row; parts without a key (LSE = -inf) are not read.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_merge_parts_kernel(const MergeParams p) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const int row = (int)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    if (row >= p.rows) return;
    const float* lse2 = p.parts.lse2 + (size_t)row * p.parts.parts;
    const float* o = p.parts.o + (size_t)row * p.parts.parts * D + lane * kPer;
    float top = -INFINITY;
    for (int i = lane; i < p.parts.parts; i += 32) top = fmaxf(top, lse2[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = 0.0f, x[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < p.parts.parts; ++i) {
        const float y = lse2[i];
        if (y == -INFINITY) continue;
        const float w = ex2_approx(y - top);
        sum += w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = fmaf(w, o[(size_t)i * D + e], x[e]);
    }
    const bool any = top != -INFINITY || sum != 0.0f;  // (a NaN part has no maximum, but a sum)
    const float f = any ? 1.0f / sum : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (size_t)row * D + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack2<BF16>(x[e] * f, x[e + 1] * f);
    if (lane == 0) p.lse[row] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D, bool Q8, bool BF16, int NT>
cudaError_t launch_t(const GqaParams& p, cudaStream_t s) {
    using C = GqaCfg<D, Q8>;
    auto kern = fa_decode_gqa_kernel<D, Q8, BF16, NT>;
    GqaParams q = p;
    q.stages = C::kStages;
    const int smem = C::smem_bytes(q.stages);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)p.splits, (unsigned)(p.Hk * p.q_blocks), (unsigned)p.B);
    return p.early ? launch_kernel_early(kern, grid, dim3(kWarps * 32), (size_t)smem, s, q)
                   : launch_kernel(kern, grid, dim3(kWarps * 32), (size_t)smem, s, q);
}

template <int D, bool Q8, bool BF16>
cudaError_t launch_n(const GqaParams& p, cudaStream_t s) {
    return p.group <= 8 ? launch_t<D, Q8, BF16, 1>(p, s) : launch_t<D, Q8, BF16, 2>(p, s);
}

template <int D>
cudaError_t launch_d(const GqaParams& p, bool bf16, bool q8, cudaStream_t s) {
    if (q8) return bf16 ? launch_n<D, true, true>(p, s) : launch_n<D, true, false>(p, s);
    return bf16 ? launch_n<D, false, true>(p, s) : launch_n<D, false, false>(p, s);
}

}  // namespace

int gqa_q_blocks(int group) { return group <= 8 ? 1 : (group + 15) / 16; }

int gqa_splits(int B, int Hk, int group, int max_pages) {
    // About four CTAs per SM of a 152-SM part (a fixed target, so that the workspace size does not
    // depend on the device), each split at least 16 pages (four per warp).
    const long long units = (long long)B * Hk * gqa_q_blocks(group);
    const long long target = 4LL * 152;
    if (units <= 0 || units >= target || max_pages <= 16) return 1;
    long long splits = (target + units - 1) / units;
    if (splits > (max_pages + 15) / 16) splits = (max_pages + 15) / 16;
    const int per = (int)((max_pages + splits - 1) / splits);
    return (max_pages + per - 1) / per;
}

cudaError_t launch_decode_gqa(const GqaParams& p, int D, bool bf16, bool q8, cudaStream_t s) {
    return D == 64 ? launch_d<64>(p, bf16, q8, s) : launch_d<128>(p, bf16, q8, s);
}

cudaError_t launch_merge_parts(const MergeParams& p, int D, bool bf16, cudaStream_t s) {
    const dim3 grid((unsigned)((p.rows + 3) / 4)), block(128);
    if (D == 64)
        return bf16 ? launch_kernel_early(fa_merge_parts_kernel<64, true>, grid, block, 0, s, p)
                    : launch_kernel_early(fa_merge_parts_kernel<64, false>, grid, block, 0, s, p);
    return bf16 ? launch_kernel_early(fa_merge_parts_kernel<128, true>, grid, block, 0, s, p)
                : launch_kernel_early(fa_merge_parts_kernel<128, false>, grid, block, 0, s, p);
}

}  // namespace fa
