// fa_prefix.cu -- all query rows of a decode batch against one shared prefix (sm_103a).
//
// Sequences that begin with the same tokens (a system prompt, a document) share those tokens' pages.
// Attending to them once per sequence would read them B times; here every cache head's prefix
// is read once and multiplied with the B * G query rows that use it:
//     S = scale Q_h K_h^T  [B G, Lp],   part (O_i, LSE_i) of every row over the prefix's tokens,
// which fa_merge_kernel joins with the part over the sequence's own tokens.
//
// 4 G B D FLOPs for 4 D bytes of a token and cache head: from B G of about 280 on the tensor cores are the
// bound, below it HBM is.  tcgen05 kernel on the plan of fa_fwd.cu: two 128-row query tiles
// share every K/V tile; TMA producer warps for K and V, one MMA warp, eight softmax warps (one row
// per thread), P as the TMEM operand of PV.  What differs:
//  * rows: row r of a tile is query g = r % G of sequence b0 + r / G, G * rows_b <= 128 of them; one
//    3-D TMA box {64, G, rows_b} of [B, Hq, D] brings them in that order.  Rows behind them hold
//    whatever the slot held: tensor-core rows do not mix, and they are not written;
//  * keys: a 128-key tile is 8 pages, each its own box of 16 rows, issued by one lane each.
//    Rows past the prefix's end must be zeros, not garbage (0 * NaN): the last page is read
//    through a map with its own row count, pages past the end at a row outside the map;
//  * split: B G rows alone seldom fill 152 SMs, so the units (head, pair of query tiles, key tile)
//    are dealt out evenly in one line over the CTAs, one per SM.  A CTA's stretch covers one or
//    more segments of pairs; each segment leaves one part per row.  Even stretches have no
//    tail (a grid of whole splits per head would idle up to half of the last wave);
//  * output: fp32 parts, each row 64 or 128 contiguous floats, staged through shared memory.
//
// 256 sequences, 32 heads of 128, a prefix of 16384 tokens: 62 us, 1108 TFLOP/s.  Doubling the prefix
// adds 43 us (1580 TFLOP/s), so that 19 do not depend on its length (start, queries, read-out).
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;
// fp16 weights are taken relative to a reference 2^7 below the largest (see fa_decode_gqa.cu).
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;
constexpr int kPagesPerTile = kTileRows / kPageTokens;
constexpr int kGrid = 152;  // CTAs at most: fixed, so that the workspace does not depend on the device

template <int D, bool BF16>
struct PrefixCfg {
    static constexpr int kChunks = D / kChunkElems;
    static constexpr int kTileBytes = kTileRows * D * 2;
    static constexpr int kStages = (D == 128) ? 2 : 4;  // of the K ring and of the V ring
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kStageBytes = 32 * 32 * 4;     // read-out buffer of one softmax warp
    static constexpr int kOffStage = kOffV + kStages * kTileBytes;
    static constexpr int kSmemBytes = kOffStage + 8 * kStageBytes + 1024;
    static constexpr int kKWarp = 8, kVWarp = 9, kMmaWarp = 10;
    static constexpr int kThreads = 11 * 32;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kTmS = 0, kTmO = 256;
    static_assert(kTmO + 2 * D <= kTmemCols, "TMEM budget");
    static_assert(kSmemBytes <= 232448, "shared memory over the 227 KB per-block limit");
    static constexpr uint32_t kIdescS = idesc_f16(BF16, 128, 128, false, false);
    static constexpr uint32_t kIdescO = idesc_f16(BF16, 128, D, false, true);
};

__host__ __device__ __forceinline__ long long cta_first_unit(long long units, int grid, int c) {
    return units * c / grid;
}
// The CTA that has unit u.
__host__ __device__ __forceinline__ int unit_cta(long long units, int grid, long long u) {
    return (int)(((u + 1) * grid - 1) / units);
}

// One segment: key tiles j0 .. j0 + n - 1 of a pair of query tiles.
struct Segment {
    int hk, pair, j0, n;
    bool has_b;
    int part;   // index of this part of the pair's rows
    bool last;  // ends the pair's key tiles
};

// The segment that begins at unit u (u < u1, the CTA's end).
__device__ __forceinline__ bool segment_at(const PrefixParams& p, long long u, long long u1,
                                           Segment& s) {
    if (u >= u1) return false;
    const long long item = u / p.key_tiles;
    s.j0 = (int)(u - item * p.key_tiles);
    s.hk = (int)(item / p.n_pairs);
    s.pair = (int)(item - (long long)s.hk * p.n_pairs);
    const long long end = (item + 1) * p.key_tiles;
    s.n = (int)((end < u1 ? end : u1) - u);
    s.has_b = 2 * s.pair + 1 < p.n_tiles;
    const long long units = (long long)p.Hk * p.n_pairs * p.key_tiles;
    s.part = (int)blockIdx.x - unit_cta(units, p.grid, item * p.key_tiles);
    s.last = end <= u1;
    return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(PrefixCfg<D, BF16>::kThreads, 1)
    fa_prefix_kernel(const __grid_constant__ PrefixParams p) {
    using C = PrefixCfg<D, BF16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    __shared__ uint64_t bar_qf, bar_qe, bar_kf[C::kStages], bar_ke[C::kStages], bar_vf[C::kStages],
        bar_ve[C::kStages], bar_sf[2], bar_pf[2], bar_oready[2], bar_fin;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_v = &abort_flag;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
        abort_flag = 0;
        mbar_init(&bar_qf, 1);
        mbar_init(&bar_qe, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar_kf[s], 1);
            mbar_init(&bar_ke[s], 1);
            mbar_init(&bar_vf[s], 1);
            mbar_init(&bar_ve[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar_sf[t], 1);
            mbar_init(&bar_pf[t], 128);
            mbar_init(&bar_oready[t], 1);
        }
        mbar_init(&bar_fin, 1);
        mbar_fence_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&tmem_base_sh, C::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    const long long units = (long long)p.Hk * p.n_pairs * p.key_tiles;
    const long long u_first = cta_first_unit(units, p.grid, (int)blockIdx.x);
    const long long u_end = cta_first_unit(units, p.grid, (int)blockIdx.x + 1);

    if (warp == C::kKWarp || warp == C::kVWarp) {
        // ------------------------------ TMA producers ------------------------------
        // The K warp also brings each segment's query pair.  Lane 8c + i issues page i of
        // chunk c; table entries are fetched one tile ahead.
        const bool is_k = warp == C::kKWarp;
        const CUtensorMap* map = is_k ? &p.tm_k : &p.tm_v;
        const CUtensorMap* map_tail = is_k ? &p.tm_k_tail : &p.tm_v_tail;
        uint64_t* full = is_k ? bar_kf : bar_vf;
        uint64_t* empty = is_k ? bar_ke : bar_ve;
        uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
        const int n_pages = (p.prefix_len + kPageTokens - 1) / kPageTokens;
        const int tail = p.prefix_len % kPageTokens;
        const int my_page = lane & (kPagesPerTile - 1), my_chunk = lane / kPagesPerTile;
        auto entry = [&](int j) {
            const int pg = j * kPagesPerTile + my_page;
            return pg < n_pages ? p.table[pg] : 0;
        };
        bool ok = true;
        int issued = 0, n_seg = 0;
        Segment sg;
        for (long long u = u_first; ok && segment_at(p, u, u_end, sg); u += sg.n) {
            int next = entry(sg.j0);
            if (is_k) {
                if (n_seg > 0) ok = wait_warp(&bar_qe, (uint32_t)(n_seg - 1) & 1u, abort_v, p.timeout_ns);
                if (!ok) break;
                if (lane == 0) {
                    const int nt = sg.has_b ? 2 : 1;
                    const uint32_t box = (uint32_t)(p.group * p.rows_b) * kChunkElems * 2;
                    mbar_arrive_expect_tx(&bar_qf, (uint32_t)nt * C::kChunks * box);
                    for (int t = 0; t < nt; ++t)
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_3d(smem + C::kOffQ + t * C::kTileBytes + c * kChunkBytes, &p.tm_q,
                                        &bar_qf, c * kChunkElems, sg.hk * p.group,
                                        (2 * sg.pair + t) * p.rows_b);
                }
                __syncwarp();
                ++n_seg;
            }
            for (int j = sg.j0; j < sg.j0 + sg.n; ++j) {
                int phys = next;
                if (j + 1 < sg.j0 + sg.n) next = entry(j + 1);
                const int st = issued % C::kStages;
                if (issued >= C::kStages) {
                    ok = wait_warp(&empty[st], ((uint32_t)(issued / C::kStages) & 1u) ^ 1u, abort_v,
                                   p.timeout_ns);
                    if (!ok) break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kTileBytes);
                __syncwarp();
                if (my_chunk < C::kChunks) {
                    const int pg = j * kPagesPerTile + my_page;
                    const CUtensorMap* m = (tail > 0 && pg == n_pages - 1) ? map_tail : map;
                    int row = 0;
                    if (pg >= n_pages) {
                        row = kPageTokens;  // outside the map: zeros
                        phys = 0;
                    } else if (phys < 0 || phys >= p.num_pages) {
                        atomicCAS(p.status, 0, (int)kDevBadArg);
                        row = kPageTokens;
                        phys = 0;
                    }
                    tma_load_3d(ring + st * C::kTileBytes + my_chunk * kChunkBytes +
                                    my_page * (kPageTokens * 128),
                                m, &full[st], my_chunk * kChunkElems, row, phys * p.Hk + sg.hk);
                }
                __syncwarp();
                ++issued;
            }
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        // Drain: the newest fill of every slot must have landed before the CTA exits.
        if (is_k && n_seg > 0)
            wait_bounded(&bar_qf, (uint32_t)(n_seg - 1) & 1u, nullptr, p.timeout_ns);
        for (int g = issued - 1; g >= 0 && g >= issued - C::kStages; --g)
            wait_bounded(&full[g % C::kStages], (uint32_t)(g / C::kStages) & 1u, nullptr, p.timeout_ns);
    } else if (warp == C::kMmaWarp) {
        // ------------------------------ MMA issuer ------------------------------
        bool ok = true;
        int g = 0, n_seg = 0, ps[2] = {0, 0};
        const uint32_t neg = p.s_negate ? kIdescNegateA : 0u;
        auto wait_ring = [&](uint64_t* full, int i) -> bool {
            const bool r = wait_warp(&full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u, abort_v,
                                     p.timeout_ns);
            tc_fence_after_sync();
            return r;
        };
        Segment sg;
        for (long long u = u_first; ok && segment_at(p, u, u_end, sg); u += sg.n) {
            const int nt = sg.has_b ? 2 : 1;
            auto issue_s = [&](int t, int gk) {  // S_t = Q_t K^T for ring fill gk
                const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + C::kOffQ + t * C::kTileBytes));
                const uint64_t kd = sdesc_kmajor_sw128(
                    smem_u32(smem + C::kOffK + (gk % C::kStages) * C::kTileBytes));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                    mma_ss_w(tmem + C::kTmS + 128 * t, sdesc_advance(qd, off), sdesc_advance(kd, off),
                             C::kIdescS | neg, kk > 0 ? 1u : 0u);
                }
                mma_commit_w(&bar_sf[t]);
            };
            auto issue_pv = [&](int t, int j) -> bool {  // O_t += P_t V_j (V_j already landed)
                if (!wait_warp(&bar_pf[t], (uint32_t)(ps[t] + j) & 1u, abort_v, p.timeout_ns))
                    return false;
                tc_fence_after_sync();
                const uint64_t vd = sdesc_mnmajor_sw128(
                    smem_u32(smem + C::kOffV + ((g + j) % C::kStages) * C::kTileBytes), kChunkBytes);
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    mma_ts_w(tmem + C::kTmO + D * t, tmem + C::kTmS + 128 * t + kk * 8,
                             sdesc_advance(vd, kk * 2048), C::kIdescO, (j > 0 || kk > 0) ? 1u : 0u);
                if (j + 1 == sg.n) mma_commit_w(&bar_oready[t]);  // O_t is final
                return true;
            };
            ok = wait_warp(&bar_qf, (uint32_t)n_seg & 1u, abort_v, p.timeout_ns);
            tc_fence_after_sync();
            ok = ok && wait_ring(bar_kf, g);
            if (!ok) break;
            for (int t = 0; t < nt; ++t) issue_s(t, g);
            if (sg.n == 1) mma_commit_w(&bar_qe);  // every S of the segment issued
            mma_commit_w(&bar_ke[g % C::kStages]);
            for (int j = 0; ok && j < sg.n; ++j) {
                const bool more = j + 1 < sg.n;
                const int gj = g + j;
                if (!wait_ring(bar_vf, gj) || (more && !wait_ring(bar_kf, gj + 1))) {
                    ok = false;
                    break;
                }
                for (int t = 0; t < nt; ++t) {
                    if (!issue_pv(t, j)) {
                        ok = false;
                        break;
                    }
                    if (more) issue_s(t, gj + 1);
                }
                if (!ok) break;
                if (j + 2 == sg.n) mma_commit_w(&bar_qe);  // the segment's last S issued
                mma_commit_w(&bar_ve[gj % C::kStages]);
                if (more) mma_commit_w(&bar_ke[(gj + 1) % C::kStages]);
            }
            g += sg.n;
            ps[0] += sg.n;
            if (nt == 2) ps[1] += sg.n;
            ++n_seg;
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        mma_commit_w(&bar_fin);  // every issued MMA must finish before TMEM is released
        wait_warp(&bar_fin, 0, nullptr, p.timeout_ns);
    } else {
        // ------------------------------ softmax warps ------------------------------
        const int t = warp / 4, quad = warp % 4;
        const int row = quad * 32 + lane;  // row inside the tile == TMEM lane
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + C::kTmS + 128 * t;
        const uint32_t o_addr = tmem + lane_off + C::kTmO + D * t;
        const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
        const uint32_t stage = smem_u32(smem + C::kOffStage + warp * C::kStageBytes);
        bool ok = true;
        int ps = 0, n_done = 0;
        Segment sg;
        for (long long u = u_first; ok && segment_at(p, u, u_end, sg); u += sg.n) {
            if (t == 1 && !sg.has_b) continue;
            float m_ref = -INFINITY, l_sum = 0.0f;
            for (int j = 0; j < sg.n; ++j) {
                ok = wait_warp(&bar_sf[t], (uint32_t)(ps + j) & 1u, abort_v, p.timeout_ns);
                if (!ok) break;
                tc_fence_after_sync();
                float s[128];
                {
                    uint32_t r[128];
                    tmem_ld_cols<128>(s_addr, r);
#pragma unroll
                    for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(r[i]);
                }
                const int left = p.prefix_len - (sg.j0 + j) * kTileRows;  // tokens from this tile on
                if (left < kTileRows) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c >= left) s[c] = -INFINITY;
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
                const bool rescale = (j > 0) && (m_new != m_ref);
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
            }
            if (!ok) break;
            ok = wait_warp(&bar_oready[t], (uint32_t)n_done & 1u, abort_v, p.timeout_ns);
            if (!ok) break;
            tc_fence_after_sync();
            // Row r of the tile: query r % G of sequence b0 + r / G.
            const int bi = row / p.group;
            const int b = (2 * sg.pair + t) * p.rows_b + bi;
            const bool valid = bi < p.rows_b && b < p.B;
            const size_t qrow = valid ? (size_t)b * p.Hq + (size_t)sg.hk * p.group + (row - bi * p.group) : 0;
            const size_t part = qrow * p.max_segments + sg.part;
            if (valid) {
                p.part_lse[part] = l_sum != 0.0f ? m_ref + log2f(l_sum) : -INFINITY;
                if (sg.last)  // parts that no CTA writes
                    for (int i = sg.part + 1; i < p.max_segments; ++i)
                        p.part_lse[qrow * p.max_segments + i] = -INFINITY;
            }
            const float inv_l = l_sum != 0.0f ? 1.0f / l_sum : 0.0f;
            // 32 columns at a time through this warp's buffer: 4 rows of 128 bytes per store.
            float* dst = valid ? p.part_o + part * D : nullptr;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                tmem_ld32(o_addr + 32 * c, r);
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    uint4 w;
                    w.x = __float_as_uint(__uint_as_float(r[4 * v + 0]) * inv_l);
                    w.y = __float_as_uint(__uint_as_float(r[4 * v + 1]) * inv_l);
                    w.z = __float_as_uint(__uint_as_float(r[4 * v + 2]) * inv_l);
                    w.w = __float_as_uint(__uint_as_float(r[4 * v + 3]) * inv_l);
                    sts_u32x4(stage + lane * 128 + ((v ^ (lane & 7)) << 4), w);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = 4 * k + (lane >> 3), uu = lane & 7;
                    const uint4 w = lds_u32x4(stage + rr * 128 + ((uu ^ (rr & 7)) << 4));
                    float* d = reinterpret_cast<float*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), rr));
                    if (d) *reinterpret_cast<uint4*>(d + c * 32 + uu * 4) = w;
                }
                __syncwarp();
            }
            ps += sg.n;
            ++n_done;
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int D, bool BF16>
cudaError_t launch_t(const PrefixParams& p, cudaStream_t s) {
    using C = PrefixCfg<D, BF16>;
    auto kern = fa_prefix_kernel<D, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmemBytes, s, p);
}

}  // namespace

void prefix_plan(int B, int Hk, int group, int prefix_len, PrefixParams* p) {
    p->rows_b = kTileRows / group;
    if (p->rows_b > B) p->rows_b = B;
    p->n_tiles = (B + p->rows_b - 1) / p->rows_b;
    p->n_pairs = (p->n_tiles + 1) / 2;
    p->key_tiles = (int)(((long long)prefix_len + kTileRows - 1) / kTileRows);
    const long long units = (long long)Hk * p->n_pairs * p->key_tiles;
    // One CTA per SM, each with four units at least (a part's read-out costs about as much, and the
    // merge reads it again; 64 sequences of up to 512 tokens behind 4096, 8 cache heads of 128: 33, 33,
    // 30, 26, 25, 27, 29 us with 1, 2, 3, 4, 5, 6, 8 units), but a quarter of the SMs at least where
    // there are so many units: a unit takes 2 us, which is all that counts in a short call.
    const long long want = (units + 3) / 4, least = units < kGrid / 4 ? units : kGrid / 4;
    p->grid = (int)(want > kGrid ? kGrid : want < least ? least : want);
    // CTAs that share one pair's key tiles: at most this many (a stretch begins every
    // units / grid units).
    p->max_segments = 0;
    if (units > 0) {
        const long long most = ((long long)p->key_tiles * p->grid + units - 1) / units + 1;
        p->max_segments = (int)(most < p->key_tiles ? most : p->key_tiles);
    }
}

cudaError_t launch_prefix(const PrefixParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_t<64, true>(p, s) : launch_t<64, false>(p, s);
    return bf16 ? launch_t<128, true>(p, s) : launch_t<128, false>(p, s);
}

}  // namespace fa
