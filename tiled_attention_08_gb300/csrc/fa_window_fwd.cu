// fa_window_fwd.cu -- attention forward under a sliding window with first tokens that stay visible,
// with grouped heads (sm_103a).
//
// Query row i (position t = i + Lk - Lq) of head h sees key j of head h / G iff 0 <= j <= t and
// (j > t - window or j < sinks); O = softmax(scale Q K^T) V over those, LSE their log-sum-exp.
//
// Bound by the tensor cores: 4 D FLOPs per visible pair and head for a few bytes of Q and O.  The
// plan is that of the dense forward: two 128-row query tiles (A, B) of 128-key tiles, K and V rings
// filled by TMA, one MMA warp, eight softmax warps (one row per thread), P as the TMEM operand of PV,
// a running reference that is raised by 2^8 steps.  What differs:
//  * key tiles: those of the first tokens, then those of the window (fa_window_sched.h); tiles that no row
//    sees are neither loaded nor multiplied, and those that every row of a warp sees whole take no mask.  (To
//    take no exponentials for 32-column pieces that none of a warp's rows sees costs more than it saves: with
//    branches between the pieces they no longer overlap, 444 -> 689 us at 8 x 4096, 32 heads, window 1024.)
//  * the pair: where a group has an even number of heads, A and B are the same query tile of two
//    of its heads, which see the same key tiles.  Else they are consecutive tiles of one head; A
//    then sits out the last key tiles and B the window's first ones.  A short call, whose single tiles find
//    an SM each, takes them one by one (the last 200 of 1500 tokens, 32 heads on 8: 20.5 -> 17.7 us).
//  * a row may see nothing in a tile that its item visits, so that its reference is still -inf there.
//
// Measured: 16384 tokens, 32 heads on 8 of 128, window 4096, 4 first tokens 640 us (1500 TFLOP/s of visible pairs);
// 8 x 4096, 32 heads of 128, window 1024 441 us (1090); 3 x 5001, 16 heads on 4 of 64, window 777, 131 first 102 us
// (497).  A step of both tiles takes 3400 cycles where its contractions take 2050: the chain from S to softmax to PV
// counts, as in the dense forward (heads of 64: tensor cores 30%, issue slots 47%, ALU 44%, XU 33%: no pipe is full
// there either).  Short windows lose the hidden halves of their first and last tiles and about 4000 cycles an item
// (first step, read-out).  Tried and dropped: S of the next item in front of this one's last PV (window 1024: 441 ->
// 435 us, others 1 to 6% slower; before the producer worked the items out 451 -> 455, and 642 -> 646 for window 4096);
// a tile of few first tokens as its first 32 keys alone (483 -> 480 us with them, 447 -> 462 without: code of two
// widths).
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_sched.h"
#include "fa_window_sched.h"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;
// fp16 weights are taken relative to a reference 2^7 below the largest, so that small ones behind a large one (a first
// token that stays visible) keep their bits: 2^-20.5 of the largest is off by eps/2, not by 2.8%.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;

template <int D, bool BF16>
struct WinCfg {
    static constexpr int kChunks = D / kChunkElems;
    static constexpr int kTileBytes = kTileRows * D * 2;
    // As in the dense forward: D = 64 one ring of K and V together and two Q slots, D = 128 a ring
    // each and one slot.
    static constexpr bool kMergedKV = (D == 64);
    static constexpr int kQSlots = (D == 128) ? 1 : 2;
    static constexpr int kStages = (D == 128) ? 2 : 4;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQSlots * 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kStageBytes = 32 * 64 * 2;  // read-out buffer of a softmax warp
    static constexpr int kOffStage = kOffV + kStages * kTileBytes;
    static constexpr int kSmemBytes = kOffStage + 8 * kStageBytes + 1024;
    static constexpr int kProducerWarp = 8, kMmaWarp = 9, kVProducerWarp = 10;
    static constexpr int kThreads = (kMergedKV ? 10 : 11) * 32;
    // The producer works the items out and leaves them in a ring of this many.  (Every warp for itself, in code that is
    // cold whenever it is reached: heads of 64, window 256 192 us against 176, window 1024 380 and 361; heads of 128,
    // window 1024 447 and 441, window 256 286 and 293.)
    static constexpr int kItems = 4;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kTmS = 0, kTmO = 256;
    static_assert(kTmO + 2 * D <= kTmemCols, "TMEM budget");
    static_assert(kSmemBytes <= 232448, "shared memory over the 227 KB per-block limit");
    static constexpr uint32_t kIdescS = idesc_f16(BF16, 128, 128, false, false);
    static constexpr uint32_t kIdescO = idesc_f16(BF16, 128, D, false, true);
};

// One work item: query tiles t = 0, 1 (tile 1 may be missing) and the key tiles that they see.
struct Item {
    int b, hk, h[2], q[2];  // batch, key head, query heads, query tiles
    KeyTiles all, of[2];
    int n, n_of[2];
};

__device__ __forceinline__ bool item_at(const WindowFwdParams& p, int round, Item& it) {
    const int id = persistent_tile(round, (int)blockIdx.x, (int)gridDim.x, p.rows * p.columns);
    if (id < 0) return false;
    int column, rank;
    tile_coords(id, p.columns, p.rows, p.sched_group, column, rank);
    const int row = p.rows - 1 - rank;  // the first rows, which may see fewer key tiles, last
    const int per_b = p.head_pairs ? p.Hq / 2 : p.Hq;
    it.b = column / per_b;
    const int c = column - it.b * per_b;
    it.h[0] = p.head_pairs ? 2 * c : c;
    it.h[1] = p.head_pairs ? 2 * c + 1 : c;
    it.hk = it.h[0] / (p.Hq / p.Hk);
    it.q[0] = p.head_pairs || p.single ? row : 2 * row;
    it.q[1] = p.head_pairs ? row : p.single ? p.Lq : 2 * row + 1;  // (Lq: no such tile)
    const int off = p.Lk - p.Lq, n_qtiles = (p.Lq + kTileRows - 1) / kTileRows;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r0 = it.q[t] * kTileRows;
        it.of[t] = it.q[t] < n_qtiles
                       ? key_tiles(r0 + off, imin(r0 + kTileRows, p.Lq) - 1 + off, p.window, p.sinks)
                       : KeyTiles{0, 0, 0};
        it.n_of[t] = it.of[t].count();
    }
    it.all = it.of[0];
    if (it.n_of[1] > 0) {  // (A's tiles begin first and B's end last; between them none is missing)
        const int r0 = it.q[0] * kTileRows;
        it.all = key_tiles(r0 + off, imin((it.q[1] + 1) * kTileRows, p.Lq) - 1 + off, p.window, p.sinks);
    }
    it.n = it.all.count();
    return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(WinCfg<D, BF16>::kThreads, 1)
    fa_window_fwd_kernel(const __grid_constant__ WindowFwdParams p) {
    using C = WinCfg<D, BF16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    __shared__ uint64_t bar_qf[C::kQSlots], bar_qe[C::kQSlots];  // Q pair landed / read by S
    __shared__ uint64_t bar_kf[C::kStages], bar_ke[C::kStages], bar_vf[C::kStages], bar_ve[C::kStages];
    __shared__ uint64_t bar_sf[2], bar_pf[2], bar_oready[2], bar_fin;
    __shared__ uint64_t bar_itf[C::kItems], bar_ite[C::kItems];  // items there / taken
    __shared__ Item item_sh[C::kItems];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_v = &abort_flag;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < C::kQSlots; ++s) {
            mbar_init(&bar_qf[s], 1);
            mbar_init(&bar_qe[s], 1);
        }
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
        for (int s = 0; s < C::kItems; ++s) {
            mbar_init(&bar_itf[s], 1);
            mbar_init(&bar_ite[s], C::kMergedKV ? 9 : 10);  // MMA, softmax and V warps
        }
        mbar_init(&bar_fin, 1);
        mbar_fence_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&tmem_base_sh, C::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    // The i-th item with a key to see, for all warps but the producer; false behind the last one, and (ok = false)
    // without it.  One of a warp's lanes may call it alone.
    auto take = [&](int i, Item& it, bool whole_warp, bool& ok) -> bool {
        const int at = i % C::kItems;
        const uint32_t ph = (uint32_t)(i / C::kItems) & 1u;
        ok = whole_warp ? wait_warp(&bar_itf[at], ph, abort_v, p.timeout_ns)
                        : wait_bounded(&bar_itf[at], ph, abort_v, p.timeout_ns);
        if (!ok) return false;
        it = item_sh[at];
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(&bar_ite[at]);
        return it.n > 0;
    };
    auto q_tile = [&](int slot, int t) { return smem + C::kOffQ + (slot * 2 + t) * C::kTileBytes; };

    if (warp == C::kProducerWarp || warp == C::kVProducerWarp) {
        // ------------------------------ TMA producers ------------------------------
        if (lane == 0) {
            const bool is_k = warp == C::kProducerWarp;
            const CUtensorMap* map = is_k ? &p.tm_k : &p.tm_v;
            uint64_t* full = is_k ? bar_kf : bar_vf;
            uint64_t* empty = is_k ? bar_ke : bar_ve;
            uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
            constexpr uint32_t kFill = (C::kMergedKV ? 2 : 1) * C::kTileBytes;
            tma_prefetch_desc(map);
            if (is_k) tma_prefetch_desc(&p.tm_q);
            if (C::kMergedKV) tma_prefetch_desc(&p.tm_v);
            bool ok = true;
            int issued = 0, n_q = 0;  // ring fills and Q pairs handed to the TMA unit
            Item it;
            int round = 0;
            // The next item, the producer: worked out and left for the others.
            auto leave = [&](int i) -> bool {
                bool more;
                while ((more = item_at(p, round++, it)) && it.n == 0) {}  // (no row sees a key)
                if (!more) it.n = 0;
                const int at = i % C::kItems;
                if (i >= C::kItems)
                    ok = wait_bounded(&bar_ite[at], (uint32_t)(i / C::kItems - 1) & 1u, abort_v, p.timeout_ns);
                if (!ok) return false;
                item_sh[at] = it;
                mbar_arrive(&bar_itf[at]);
                return more;
            };
            for (int i = 0; ok && (is_k ? leave(i) : take(i, it, false, ok)); ++i) {
                if (is_k) {
                    const int qs = n_q % C::kQSlots, use = n_q / C::kQSlots;
                    if (use > 0 && !wait_bounded(&bar_qe[qs], (uint32_t)(use - 1) & 1u, abort_v, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bar_qf[qs],
                                          ((it.n_of[0] > 0) + (it.n_of[1] > 0)) * (uint32_t)C::kTileBytes);
                    for (int t = 0; t < 2; ++t)
                        for (int c = 0; it.n_of[t] > 0 && c < C::kChunks; ++c)
                            tma_load_4d(q_tile(qs, t) + c * kChunkBytes, &p.tm_q, &bar_qf[qs], c * kChunkElems,
                                        it.q[t] * kTileRows, it.h[t], it.b);
                    ++n_q;
                }
                for (int j = 0; j < it.n; ++j) {
                    const int st = issued % C::kStages;
                    const uint32_t ph = (uint32_t)(issued / C::kStages) & 1u;
                    if (issued >= C::kStages && !wait_bounded(&empty[st], ph ^ 1u, abort_v, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const int key0 = it.all.tile(j) * kTileRows;
                    mbar_arrive_expect_tx(&full[st], kFill);
                    for (int c = 0; c < C::kChunks; ++c) {
                        tma_load_4d(ring + st * C::kTileBytes + c * kChunkBytes, map, &full[st],
                                    c * kChunkElems, key0, it.hk, it.b);
                        if constexpr (C::kMergedKV)
                            tma_load_4d(smem + C::kOffV + st * C::kTileBytes + c * kChunkBytes, &p.tm_v,
                                        &full[st], c * kChunkElems, key0, it.hk, it.b);
                    }
                    ++issued;
                }
            }
            if (!ok) record_timeout(p.status, abort_v);
            // Drain: the newest fill of every slot must have landed before the CTA exits.
            for (int n = n_q - 1; n >= 0 && n >= n_q - C::kQSlots; --n)
                wait_bounded(&bar_qf[n % C::kQSlots], (uint32_t)(n / C::kQSlots) & 1u, nullptr, p.timeout_ns);
            for (int g = issued - 1; g >= 0 && g >= issued - C::kStages; --g)
                wait_bounded(&full[g % C::kStages], (uint32_t)(g / C::kStages) & 1u, nullptr, p.timeout_ns);
        }
    } else if (warp == C::kMmaWarp) {
        // ------------------------------ MMA issuer ------------------------------
        // g counts ring fills, ps[t] the S / P completions of tile t, over the CTA's lifetime.  S_t of
        // the next key tile is issued behind PV_t, so it never overwrites a P still being read.
        bool ok = true;
        int g = 0, n_item = 0, ps[2] = {0, 0}, k_ready = -1;
        auto wait_k = [&](int gk) -> bool {
            if (k_ready >= gk) return true;
            if (!wait_warp(&bar_kf[gk % C::kStages], (uint32_t)(gk / C::kStages) & 1u, abort_v, p.timeout_ns))
                return false;
            tc_fence_after_sync();
            k_ready = gk;
            return true;
        };
        Item it;
        for (int i = 0; ok && take(i, it, true, ok); ++i) {
            const int qs = n_item % C::kQSlots;
            int done[2] = {0, 0};  // PV of tile t in this item
            auto issue_s = [&](int t, int gk) {  // S_t = Q_t K^T for ring fill gk
                const uint64_t qd = sdesc_kmajor_sw128(smem_u32(q_tile(qs, t)));
                const uint64_t kd =
                    sdesc_kmajor_sw128(smem_u32(smem + C::kOffK + (gk % C::kStages) * C::kTileBytes));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                    mma_ss_w(tmem + C::kTmS + 128 * t, sdesc_advance(qd, off), sdesc_advance(kd, off),
                             C::kIdescS | p.s_negate, kk > 0 ? 1u : 0u);
                }
                mma_commit_w(&bar_sf[t]);
            };
            auto issue_pv = [&](int t, int gv) -> bool {  // O_t += P_t V for ring fill gv (landed)
                if (!wait_warp(&bar_pf[t], (uint32_t)ps[t] & 1u, abort_v, p.timeout_ns)) return false;
                tc_fence_after_sync();
                const uint64_t vd = sdesc_mnmajor_sw128(
                    smem_u32(smem + C::kOffV + (gv % C::kStages) * C::kTileBytes), kChunkBytes);
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    mma_ts_w(tmem + C::kTmO + D * t, tmem + C::kTmS + 128 * t + kk * 8,
                             sdesc_advance(vd, kk * 2048), C::kIdescO, (done[t] > 0 || kk > 0) ? 1u : 0u);
                ++ps[t];
                if (++done[t] == it.n_of[t]) mma_commit_w(&bar_oready[t]);  // O_t is final
                return true;
            };
            ok = wait_warp(&bar_qf[qs], (uint32_t)(n_item / C::kQSlots) & 1u, abort_v, p.timeout_ns);
            tc_fence_after_sync();
            ok = ok && wait_k(g);
            if (!ok) break;
            int kt = it.all.tile(0);
            for (int t = 0; t < 2; ++t)
                if (it.of[t].has(kt)) issue_s(t, g);
            if (it.n == 1) mma_commit_w(&bar_qe[qs]);  // every S of the item issued
            if constexpr (!C::kMergedKV) mma_commit_w(&bar_ke[g % C::kStages]);  // K_0 read
            for (int j = 0; ok && j < it.n; ++j) {
                const bool next = j + 1 < it.n;
                const int gj = g + j, kn = it.all.tile(j + 1);
                if constexpr (!C::kMergedKV) {
                    ok = wait_warp(&bar_vf[gj % C::kStages], (uint32_t)(gj / C::kStages) & 1u, abort_v,
                                   p.timeout_ns);
                    tc_fence_after_sync();
                }
                if (!ok || (next && !wait_k(gj + 1))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok) break;
                    if (it.of[t].has(kt) && !issue_pv(t, gj)) {
                        ok = false;
                        break;
                    }
                    if (next && it.of[t].has(kn)) issue_s(t, gj + 1);
                }
                if (!ok) break;
                if (j + 2 == it.n) mma_commit_w(&bar_qe[qs]);  // the item's last S issued
                if constexpr (C::kMergedKV) {
                    mma_commit_w(&bar_ke[gj % C::kStages]);  // K_j and V_j read
                } else {
                    mma_commit_w(&bar_ve[gj % C::kStages]);
                    if (next) mma_commit_w(&bar_ke[(gj + 1) % C::kStages]);
                }
                kt = kn;
            }
            g += it.n;
            ++n_item;
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        mma_commit_w(&bar_fin);  // every issued MMA must finish before TMEM is released
        wait_warp(&bar_fin, 0, nullptr, p.timeout_ns);
    } else {
        // ------------------------------ softmax warps ------------------------------
        const int t = warp / 4, quad = warp % 4;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + C::kTmS + 128 * t;
        const uint32_t o_addr = tmem + lane_off + C::kTmO + D * t;
        const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
        bool ok = true;
        int ps = 0, n_done = 0;
        Item it;
        for (int i = 0; ok && take(i, it, true, ok); ++i) {
            const KeyTiles mine = t ? it.of[1] : it.of[0];
            const int n = mine.count();
            if (n == 0) continue;
            const int row0 = (t ? it.q[1] : it.q[0]) * kTileRows + quad * 32;  // the warp's first row
            const int first = row0 + (p.Lk - p.Lq), pos = first + lane;        // positions
            float m_ref = -INFINITY, l_sum = 0.0f;
            for (int j = 0; j < n; ++j) {
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
                const int key0 = mine.tile(j) * kTileRows;
                // (rows past Lq see keys past Lk, which read as zeros; they are not written)
                const bool later = hides_later(key0, kTileRows, first);
                const bool earlier = hides_earlier(key0, kTileRows, first + 31, p.window, p.sinks);
                if (later) {
                    const int lim = pos - key0;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > lim) s[c] = -INFINITY;
                }
                if (earlier) {
                    const int lim = pos - p.window - key0, sink = p.sinks - key0;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c <= lim && c >= sink) s[c] = -INFINITY;
                }
                float m4[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) m4[u] = fmaxf(s[u], s[u + 4]);
#pragma unroll
                for (int c = 8; c < 128; c += 8) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) m4[u] = fmax3(m4[u], s[c + u], s[c + 4 + u]);
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
                // S_t was issued behind the last PV_t, so every PV into O_t has completed.
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
            const int bh = it.b * p.Hq + (t ? it.h[1] : it.h[0]);
            if (row0 + lane < p.Lq)
                p.lse[(size_t)bh * p.Lq + row0 + lane] =
                    l_sum != 0.0f ? (m_ref + log2f(l_sum)) * kLn2 : -INFINITY;
            // The read-out finishes before this group publishes P of the next item, which is what
            // lets PV overwrite O_t.
            const float inv_l = l_sum != 0.0f ? 1.0f / l_sum : 0.0f;
            tmem_rows_to_global_staged<BF16, D>(
                o_addr, smem_u32(smem + C::kOffStage + warp * C::kStageBytes),
                reinterpret_cast<uint8_t*>(p.o) + row_offset(p.so, bh, p.Hq, row0), (size_t)p.so.l * 2u,
                p.Lq - row0, inv_l, lane);
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
cudaError_t launch_t(const WindowFwdParams& p, cudaStream_t s) {
    using C = WinCfg<D, BF16>;
    constexpr auto kern = fa_window_fwd_kernel<D, BF16>;
    const cudaError_t e = allow_shared_once<kern>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int total = p.rows * p.columns, sms = sm_count();
    const int grid = sms > 0 && sms < total ? sms : total;
    return launch_kernel(kern, dim3((unsigned)grid), dim3(C::kThreads), C::kSmemBytes, s, p);
}

}  // namespace

cudaError_t launch_window_fwd(const WindowFwdParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_t<64, true>(p, s) : launch_t<64, false>(p, s);
    return bf16 ? launch_t<128, true>(p, s) : launch_t<128, false>(p, s);
}

}  // namespace fa
