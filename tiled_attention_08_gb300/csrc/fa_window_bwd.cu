// fa_window_bwd.cu -- backward of attention under a sliding window with first tokens that stay
// visible, with grouped heads (sm_103a).
//
// With P = exp(S - LSE) over the visible entries (fa_window_fwd.cu) and dP = dO V^T,
//     dS = P o (dP - Delta),  dQ_h = scale dS_h K,
//     dK = scale sum_h dS_h^T Q_h,  dV = sum_h P_h^T dO_h   over the heads h of the key head's group.
// Two passes on the plan of the dense backward's persistent kernels, deterministic: dK and dV per
// (key tile, key head), dQ per (query tile, head); both recompute P from the saved LSE.  Before them Delta, from O
// and dO (the dense backward's preprocess) and for rows of few keys from P and dP.  The pipelines,
// barriers and TMEM layouts are those described there.  Bound by the tensor cores: 10 D FLOPs per
// visible pair and head, 14 with the recomputed S and dP.  What differs:
//  * a dK/dV item's units are the query tiles of all heads of the group that see its key tile, head
//    after head: the sum over shared heads stays in the TMEM accumulators, with no atomics.
//  * the tiles of the first tokens are seen by every later query tile: one CTA alone would still be
//    busy when all others have finished.  Where it would, their units are cut into parts of a window
//    item's size, left as fp32 and joined in a fixed order by a third kernel.
//  * key tiles that no query sees get zeros.
//
// Measured (dK/dV, dQ, all): 16384 tokens, 32 heads on 8 of 128, window 4096, 4 first tokens 1311, 878, 2260 us (1070
// TFLOP/s of 10 D FLOPs, 1490 of the 14 D executed); 8 x 4096, 32 heads of 128, window 1024 829, 632, 1580 us (760);
// 3 x 5001, 16 heads on 4 of 64, window 777, 131 first tokens 186, 135, 362 us (350).  Tried and dropped: the last key
// tiles of all heads taken last, for an evener end (1311 -> 1294 us, but 383 -> 393 at heads of 64, which spill).
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_queue.cuh"
#include "fa_sched.h"
#include "fa_window_sched.h"

namespace fa {
namespace {

template <int D, bool BF16>
struct DkdvCfg {
    static constexpr int kChunks = D / kChunkElems;
    static constexpr int kTileBytes = kTileRows * D * 2;
    static constexpr int kQStages = (D == 128) ? 3 : 5;  // Q is needed early (S^T) and late (dK)
    static constexpr int kOStages = (D == 128) ? 2 : 4;
    static constexpr int kKVSlots = (D == 128) ? 1 : 2;
    static constexpr int kVecBytes = kTileRows * 4;  // one fp32 vector of a 128-row tile
    static constexpr int kOffK = 0;                  // slot s: K at kOffK + 2*s*kTileBytes, then V
    static constexpr int kOffQ = 2 * kKVSlots * kTileBytes;
    static constexpr int kOffDO = kOffQ + kQStages * kTileBytes;
    static constexpr int kOffNlse = kOffDO + kOStages * kTileBytes;    // per Q slot
    static constexpr int kOffDelta = kOffNlse + kQStages * kVecBytes;  // per dO slot
    static constexpr int kOffBar = kOffDelta + kOStages * kVecBytes;
    static constexpr int kSplit = 4;  // elementwise warps per TMEM lane quadrant
    static constexpr int kEwWarps = 4 * kSplit;
    static constexpr int kEwThreads = kEwWarps * 32;
    static constexpr int kProducerWarp = kEwWarps;
    static constexpr int kMmaWarp = kEwWarps + 1;
    static constexpr int kThreads = (kEwWarps + 2) * 32;
    static constexpr int kCols = 128 / kSplit;   // query columns per elementwise warp
    static constexpr int kOutCols = D / kSplit;  // dK/dV columns per elementwise warp
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kTmST = 0, kTmDPT = 128, kTmDV = 256, kTmDK = 256 + D;
    static constexpr uint32_t kIdescS = idesc_f16(BF16, 128, 128, false, false);
    static constexpr uint32_t kIdescG = idesc_f16(BF16, 128, D, false, true);
};

// Barriers and small shared state, placed after the tiles in dynamic shared memory.
template <int KVS, int QS, int OS>
struct DkdvBars {
    uint64_t kvf[KVS], kve[KVS], qf[QS], qe[QS], of[OS], oe[OS], sf, df, sr, ppd, done, fin;
    WorkQueue queue;
    uint32_t tmem_base;
    int abort;
};
template <int D, bool BF16>
using DkdvBarsT = DkdvBars<DkdvCfg<D, BF16>::kKVSlots, DkdvCfg<D, BF16>::kQStages, DkdvCfg<D, BF16>::kOStages>;

// A work item: units first .. of key tile kt of key head hk; a unit is a query tile of a head.
struct DkdvItem;
struct Unit {
    int h, qi;
    __device__ __forceinline__ void step(const DkdvItem& it);
};
struct DkdvItem {
    int b, hk, kt, n_it;
    int part;  // index of its fp32 part, or -1: it writes dK and dV
    QueryTiles q;
    Unit first;
};
__device__ __forceinline__ void Unit::step(const DkdvItem& it) {
    if (++qi == it.q.hi) {
        qi = it.q.lo;
        ++h;
    }
}

// Rows that see fewer keys than this get their Delta from P and dP (fa_window_dq_kernel): the error that O's
// rounding would leave there falls with the keys, and is 1% of dS's own from here on.
constexpr int kDeltaKeys = 256;

// Units u0 .. u1 - 1 of part i of n.
__host__ __device__ __forceinline__ int part_start(int units, int i, int n) {
    return (int)((long long)units * i / n);
}

__device__ __forceinline__ void dkdv_item(const WindowBwdParams& p, int id, DkdvItem& it) {
    const int heads = p.B * p.Hk, cut = heads * p.split_tiles * p.parts;
    int bhk, i = 0, n = 1;
    it.part = -1;
    if (id < cut) {  // the first tokens' tiles (or their parts) first: none is smaller than a window's item
        const int rest = id / heads;
        bhk = id - rest * heads;
        it.kt = rest / p.parts;
        i = rest - it.kt * p.parts;
        n = p.parts;
        if (n > 1) it.part = (bhk * p.split_tiles + it.kt) * p.parts + i;
    } else {
        tile_coords(id - cut, heads, p.n_ktiles - p.split_tiles, p.sched_group_k, bhk, it.kt);
        it.kt += p.split_tiles;
    }
    it.b = bhk / p.Hk;
    it.hk = bhk - it.b * p.Hk;
    const int group = p.Hq / p.Hk;
    it.q = query_tiles(it.kt, p.Lq, p.Lk - p.Lq, p.window, p.sinks);
    const int per_head = it.q.hi - it.q.lo, units = per_head * group;
    const int u0 = part_start(units, i, n);
    it.n_it = part_start(units, i + 1, n) - u0;
    const int g = per_head > 0 ? u0 / per_head : 0;
    it.first.h = it.hk * group + g;
    it.first.qi = it.q.lo + u0 - g * per_head;
}

// This thread's row of N accumulator columns (from column N * slice on) into an fp32 part, whose groups
// of four columns lie together for all 128 rows, so that a warp's stores are contiguous.
template <int N>
__device__ __forceinline__ void part_out(uint32_t taddr, float* dst, int slice, int row) {
    float4* d = reinterpret_cast<float4*>(dst) + (size_t)slice * (N / 4) * kTileRows + row;
#pragma unroll 1
    for (int h = 0; h < N; h += 16) {
        uint32_t r[16];
        tmem_ld16(taddr + h, r);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            d[(size_t)(h / 4 + c) * kTileRows] =
                make_float4(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1]),
                            __uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3]));
    }
}

// dK and dV.
template <int D, bool BF16>
__global__ void __launch_bounds__(DkdvCfg<D, BF16>::kThreads, 1)
    fa_window_dkdv_kernel(const __grid_constant__ WindowBwdParams p) {
    using C = DkdvCfg<D, BF16>;
    // The kernel declares no static shared memory, so its dynamic shared memory starts at the
    // block's shared window, which is 1024-byte aligned; checked here (the 128-byte swizzle
    // needs it) before any barrier, TMEM or copy is touched.
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, (int)kDevBadShared);  // -> FA_ERR_CUDA
        return;
    }
    // Q_i (+ LSE_i) and dO_i (+ Delta_i) have their own rings and full/empty barriers: Q_i is
    // released by dK_i, issued first, so the load of a later Q tile (needed early, by S^T)
    // starts sooner.
    auto& bars = *reinterpret_cast<DkdvBarsT<D, BF16>*>(smem + C::kOffBar);
    uint64_t* bar_kvf = bars.kvf;
    uint64_t* bar_kve = bars.kve;
    uint64_t* bar_qf = bars.qf;
    uint64_t* bar_qe = bars.qe;
    uint64_t* bar_of = bars.of;
    uint64_t* bar_oe = bars.oe;
    uint64_t& bar_sf = bars.sf;
    uint64_t& bar_df = bars.df;
    uint64_t& bar_sr = bars.sr;
    uint64_t& bar_ppd = bars.ppd;
    uint64_t& bar_done = bars.done;
    uint64_t& bar_fin = bars.fin;
    uint32_t& tmem_base_sh = bars.tmem_base;
    int& abort_flag = bars.abort;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    volatile int* abort_v = &abort_flag;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < C::kKVSlots; ++s) {
            mbar_init(&bar_kvf[s], 1);
            mbar_init(&bar_kve[s], 1);
        }
        for (int s = 0; s < C::kQStages; ++s) {
            mbar_init(&bar_qf[s], 1);
            mbar_init(&bar_qe[s], 1);
        }
        for (int s = 0; s < C::kOStages; ++s) {
            mbar_init(&bar_of[s], 1);
            mbar_init(&bar_oe[s], 1);
        }
        mbar_init(&bar_sf, 1);
        mbar_init(&bar_df, 1);
        mbar_init(&bar_sr, C::kEwThreads);   // S^T read: its columns may be overwritten
        mbar_init(&bar_ppd, C::kEwThreads);  // P^T and dS^T written into the dP^T columns
        mbar_init(&bar_done, 1);             // every MMA of an item complete: dK, dV final
        mbar_init(&bar_fin, 1);
        queue_init(bars.queue, 1 + C::kEwWarps);  // read by the MMA and elementwise warps
        mbar_fence_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&tmem_base_sh, C::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base_sh;
    auto k_tile = [&](int slot) { return smem + C::kOffK + 2 * slot * C::kTileBytes; };
    auto v_tile = [&](int slot) { return smem + C::kOffK + (2 * slot + 1) * C::kTileBytes; };

    if (warp == C::kProducerWarp) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            tma_prefetch_desc(&p.tm_q);
            tma_prefetch_desc(&p.tm_k);
            tma_prefetch_desc(&p.tm_v);
            tma_prefetch_desc(&p.tm_do);
            bool ok = true;
            int issued_kv = 0, issued_q = 0, issued_o = 0;
            // Q_u and -LSE*log2e into Q slot u % kQStages (u counts units over the CTA's lifetime).
            auto load_q = [&](int u, const DkdvItem& it, const Unit& n) -> bool {
                const int st = u % C::kQStages;
                if (u >= C::kQStages &&
                    !wait_bounded(&bar_qe[st], ((uint32_t)(u / C::kQStages) & 1u) ^ 1u, abort_v,
                                  p.timeout_ns))
                    return false;
                mbar_arrive_expect_tx(&bar_qf[st], C::kTileBytes + C::kVecBytes);
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load_4d(smem + C::kOffQ + st * C::kTileBytes + c * kChunkBytes, &p.tm_q,
                                &bar_qf[st], c * kChunkElems, n.qi * kTileRows, n.h, it.b);
                bulk_load(smem + C::kOffNlse + st * C::kVecBytes,
                          p.nlse2_pad + ((size_t)it.b * p.Hq + n.h) * p.Lqpad + (size_t)n.qi * kTileRows,
                          C::kVecBytes,
                          &bar_qf[st]);
                issued_q = u + 1;
                return true;
            };
            auto load_do = [&](int u, const DkdvItem& it, const Unit& n) -> bool {  // dO_u, Delta_u
                const int st = u % C::kOStages;
                if (u >= C::kOStages &&
                    !wait_bounded(&bar_oe[st], ((uint32_t)(u / C::kOStages) & 1u) ^ 1u, abort_v,
                                  p.timeout_ns))
                    return false;
                mbar_arrive_expect_tx(&bar_of[st], C::kTileBytes + C::kVecBytes);
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load_4d(smem + C::kOffDO + st * C::kTileBytes + c * kChunkBytes, &p.tm_do,
                                &bar_of[st], c * kChunkElems, n.qi * kTileRows, n.h, it.b);
                bulk_load(smem + C::kOffDelta + st * C::kVecBytes,
                          p.delta_pad + ((size_t)it.b * p.Hq + n.h) * p.Lqpad + (size_t)n.qi * kTileRows,
                          C::kVecBytes,
                          &bar_of[st]);
                issued_o = u + 1;
                return true;
            };
            int u = 0;
            DkdvItem it;
            // Item ids are fetched one round ahead of the loads (fa_queue.cuh).
            int next_id = queue_push(bars.queue, 0, p.sched, p.dkdv_items, false, abort_v,
                                     p.timeout_ns);
            for (int round = 0; ok; ++round) {
                const int id = next_id;
                if (id == -2) ok = false;
                if (id < 0) break;
                next_id = queue_push(bars.queue, round + 1, p.sched, p.dkdv_items, false,
                                     abort_v, p.timeout_ns);
                dkdv_item(p, id, it);
                if (it.n_it == 0) continue;  // no query sees the tile: its zeros are written below
                // K_j and V_j into K/V slot n_kv % kKVSlots, once the item that used it last has
                // completed its S^T and dP^T contractions.
                const int kvs = issued_kv % C::kKVSlots;
                const int use = issued_kv / C::kKVSlots;
                if (use > 0 && !wait_bounded(&bar_kve[kvs], (uint32_t)(use - 1) & 1u, abort_v,
                                             p.timeout_ns)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&bar_kvf[kvs], 2 * C::kTileBytes);
                for (int c = 0; c < C::kChunks; ++c) {
                    tma_load_4d(k_tile(kvs) + c * kChunkBytes, &p.tm_k, &bar_kvf[kvs],
                                c * kChunkElems, it.kt * kTileRows, it.hk, it.b);
                    tma_load_4d(v_tile(kvs) + c * kChunkBytes, &p.tm_v, &bar_kvf[kvs],
                                c * kChunkElems, it.kt * kTileRows, it.hk, it.b);
                }
                ++issued_kv;
                // Q runs one tile ahead of dO: Q_{t+1} only waits for dK_{t+1-kQStages}.
                Unit n = it.first;
                ok = load_q(u, it, n);
                for (int t = 0; ok && t < it.n_it; ++t) {
                    const Unit here = n;
                    n.step(it);
                    if (t + 1 < it.n_it) ok = load_q(u + t + 1, it, n);
                    ok = ok && load_do(u + t, it, here);
                }
                u += it.n_it;
            }
            if (!ok) record_timeout(p.status, abort_v);
            // Drain: no copy may still be landing when the CTA exits.
            for (int n = issued_kv - 1; n >= 0 && n >= issued_kv - C::kKVSlots; --n)
                wait_bounded(&bar_kvf[n % C::kKVSlots], (uint32_t)(n / C::kKVSlots) & 1u, nullptr,
                             p.timeout_ns);
            for (int t = issued_q - 1; t >= 0 && t >= issued_q - C::kQStages; --t)
                wait_bounded(&bar_qf[t % C::kQStages], (uint32_t)(t / C::kQStages) & 1u, nullptr,
                             p.timeout_ns);
            for (int t = issued_o - 1; t >= 0 && t >= issued_o - C::kOStages; --t)
                wait_bounded(&bar_of[t % C::kOStages], (uint32_t)(t / C::kOStages) & 1u, nullptr,
                             p.timeout_ns);
        }
    } else if (warp == C::kMmaWarp) {
        // ------------------------------ MMA issuer ------------------------------
        // The whole warp walks the loop (warp-uniform values); one elected lane issues.  u counts
        // query tiles over the CTA's lifetime (ring slots and the per-tile barrier phases).
        auto q_base = [&](int uu) {
            return smem_u32(smem + C::kOffQ + (uu % C::kQStages) * C::kTileBytes);
        };
        auto do_base = [&](int uu) {
            return smem_u32(smem + C::kOffDO + (uu % C::kOStages) * C::kTileBytes);
        };
        auto wait_q = [&](int uu) {  // Q_uu landed
            const bool r = wait_warp(&bar_qf[uu % C::kQStages], (uint32_t)(uu / C::kQStages) & 1u,
                                     abort_v, p.timeout_ns);
            tc_fence_after_sync();
            return r;
        };
        auto wait_do = [&](int uu) {  // dO_uu landed
            const bool r = wait_warp(&bar_of[uu % C::kOStages], (uint32_t)(uu / C::kOStages) & 1u,
                                     abort_v, p.timeout_ns);
            tc_fence_after_sync();
            return r;
        };
        bool ok = true;
        int u = 0, n_kv = 0;  // units, and items with any
        DkdvItem it;
        for (int round = 0; ok; ++round) {
            const int id = queue_pop_warp(bars.queue, round, abort_v, p.timeout_ns);
            if (id == -2) ok = false;
            if (id < 0) break;
            dkdv_item(p, id, it);
            if (it.n_it == 0) continue;
            const int kvs = n_kv % C::kKVSlots;
            const int n = it.n_it;
            const uint64_t kdesc = sdesc_kmajor_sw128(smem_u32(k_tile(kvs)));
            const uint64_t vdesc = sdesc_kmajor_sw128(smem_u32(v_tile(kvs)));
            auto issue_st = [&](int uu) {  // S^T = K Q_uu^T
                const uint64_t qd = sdesc_kmajor_sw128(q_base(uu));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                    mma_ss_w(tmem + C::kTmST, sdesc_advance(kdesc, off), sdesc_advance(qd, off),
                             C::kIdescS, kk > 0 ? 1u : 0u);
                }
                mma_commit_w(&bar_sf);
            };
            auto issue_dpt = [&](int uu) {  // dP^T = V dO_uu^T
                const uint64_t dd = sdesc_kmajor_sw128(do_base(uu));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                    mma_ss_w(tmem + C::kTmDPT, sdesc_advance(vdesc, off), sdesc_advance(dd, off),
                             C::kIdescS, kk > 0 ? 1u : 0u);
                }
                mma_commit_w(&bar_df);
            };
            // K_j / V_j of this item landed; the previous item's last S^T has been read (its
            // columns are reused).  The dP^T columns were last read by the previous item's last
            // dK / dV, issued before this point.
            ok = wait_warp(&bar_kvf[kvs], (uint32_t)(n_kv / C::kKVSlots) & 1u, abort_v,
                           p.timeout_ns);
            ++n_kv;
            if (ok && u > 0) ok = wait_warp(&bar_sr, (uint32_t)(u - 1) & 1u, abort_v, p.timeout_ns);
            ok = ok && wait_q(u);
            if (!ok) break;
            issue_st(u);
            if (!wait_do(u)) {
                ok = false;
                break;
            }
            issue_dpt(u);
            if (n == 1) mma_commit_w(&bar_kve[kvs]);  // the item's only S^T and dP^T issued
            for (int t = 0; t < n && ok; ++t) {
                const int uu = u + t;
                const uint32_t par = (uint32_t)uu & 1u;
                if (t + 1 < n) {
                    // S^T of the next query tile as soon as this one's S^T has been read.
                    if (!wait_warp(&bar_sr, par, abort_v, p.timeout_ns) || !wait_q(uu + 1)) {
                        ok = false;
                        break;
                    }
                    issue_st(uu + 1);
                }
                // With three or more dO slots, dO_{t+1} has normally landed by now: wait for it
                // here so dK_t, dV_t and dP^T_{t+1} go out as one batch.  With two it may still
                // be in flight, and waiting here would hold up dK_t and dV_t (measured slower).
                constexpr bool kEarlyDo = C::kOStages >= 3;
                if ((kEarlyDo && t + 1 < n && !wait_do(uu + 1)) ||
                    !wait_warp(&bar_ppd, par, abort_v, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t acc0 = t > 0 ? 1u : 0u;
                const uint64_t dod = sdesc_mnmajor_sw128(do_base(uu), kChunkBytes);
                const uint64_t qmd = sdesc_mnmajor_sw128(q_base(uu), kChunkBytes);
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    mma_ts_w(tmem + C::kTmDK, tmem + C::kTmDPT + 64 + kk * 8,
                             sdesc_advance(qmd, kk * 2048), C::kIdescG, (acc0 || kk > 0) ? 1u : 0u);
                mma_commit_w(&bar_qe[uu % C::kQStages]);  // Q_t fully read
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    mma_ts_w(tmem + C::kTmDV, tmem + C::kTmDPT + kk * 8,
                             sdesc_advance(dod, kk * 2048), C::kIdescG, (acc0 || kk > 0) ? 1u : 0u);
                mma_commit_w(&bar_oe[uu % C::kOStages]);  // dO_t fully read
                if (t + 1 < n) {  // after dV_t, dK_t read the dP^T columns
                    if (!kEarlyDo && !wait_do(uu + 1)) {
                        ok = false;
                        break;
                    }
                    issue_dpt(uu + 1);
                    if (t + 2 == n) mma_commit_w(&bar_kve[kvs]);  // the item's last S^T, dP^T
                }
            }
            if (!ok) break;
            mma_commit_w(&bar_done);
            u += n;
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        mma_commit_w(&bar_fin);
        wait_warp(&bar_fin, 0, nullptr, p.timeout_ns);
    } else {
        // ------------------------------ elementwise warps ------------------------------
        constexpr int kC = C::kCols;
        const int quad = warp & 3;              // TMEM lane quadrant (key rows)
        const int part = warp >> 2;             // which kC query columns
        const uint32_t grp_bar = 1 + quad;      // named barrier of the quadrant
        constexpr uint32_t kGrpThreads = 32 * C::kSplit;
        const int row = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const int c0 = part * kC;
        const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
        bool ok = true;
        int u = 0;                 // query tiles of earlier items
        uint32_t done_par = 0u;    // phase of the item's done barrier
        for (int round = 0; ok; ++round) {
            // The quadrant's warps agree on the outcome before any of them goes on: they meet
            // at named barriers below.
            int id = queue_pop_warp(bars.queue, round, abort_v, p.timeout_ns);
            ok = bar_and(grp_bar, kGrpThreads, id != -2);
            if (!ok || id < 0) break;
            // The loop is at the limit of 96 registers: it keeps of the item no more than it needs, in units
            // of the tile's key offset (keys and positions relative to the tile's first query row).
            int key, qi, q_lo, q_hi, u_end;
            {
                DkdvItem it;
                dkdv_item(p, id, it);
                key = it.kt * kTileRows + row;
                qi = it.first.qi;
                q_lo = it.q.lo;
                q_hi = it.q.hi;
                u_end = u + it.n_it;
            }
            const bool empty = u_end == u;
            for (; u < u_end; ++u) {
                const int uu = u;
                const int qs = uu % C::kQStages, os = uu % C::kOStages;  // ring slots of Q, dO
                const uint32_t qph = (uint32_t)(uu / C::kQStages) & 1u;
                const uint32_t oph = (uint32_t)(uu / C::kOStages) & 1u;
                // -LSE*log2e and Delta of this warp's query columns (broadcast shared reads).
                const uint32_t nlse2_addr =
                    smem_u32(smem + C::kOffNlse + qs * C::kVecBytes) + c0 * 4;
                const uint32_t dlt_addr = smem_u32(smem + C::kOffDelta + os * C::kVecBytes) + c0 * 4;
                // This warp's first query row, and its position; a query at position t sees this thread's
                // key iff key <= t < key + window, or t >= key for a first token.
                const int q0 = qi * kTileRows + c0, t0 = q0 + (p.Lk - p.Lq);
                if (++qi == q_hi) qi = q_lo;
                const bool masked = hides_later(key - lane, 32, t0) || q0 + kC > p.Lq ||
                                    hides_earlier(key - lane, 32, t0 + kC - 1, p.window, p.sinks);
                // Phase 1: P^T = exp2(S^T * scale*log2e - LSE*log2e) on this warp's columns;
                // kept in registers, and the S^T columns are released at once.
                ok = wait_bounded(&bar_qf[qs], qph, abort_v, p.timeout_ns) &&
                     wait_bounded(&bar_sf, (uint32_t)uu & 1u, abort_v, p.timeout_ns);
                ok = __all_sync(0xffffffffu, ok);
                float pv[kC];
                uint32_t pk_p[kC / 2];  // P^T, packed to 16 bits
                if (ok) {
                    tc_fence_after_sync();
                    uint32_t r[kC];
                    tmem_ld_cols<kC>(tmem + lane_off + C::kTmST + c0, r);
                    tc_fence_before_sync();
                    mbar_arrive(&bar_sr);
#pragma unroll
                    for (int i = 0; i < kC; i += 4) {  // two columns per f32x2 instruction
                        const float4 l = lds_f32x4(nlse2_addr + i * 4);
                        float y0, y1, y2, y3;
                        f2_split(f2_fma(f2_make(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                        scale2, f2_make(l.x, l.y)),
                                 y0, y1);
                        f2_split(f2_fma(f2_make(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])),
                                        scale2, f2_make(l.z, l.w)),
                                 y2, y3);
                        pv[i + 0] = ex2_approx(y0);
                        pv[i + 1] = ex2_approx(y1);
                        pv[i + 2] = ex2_approx(y2);
                        pv[i + 3] = ex2_approx(y3);
                    }
                    if (masked) {
                        const int from = key - t0;
                        const int until = imin(key < p.sinks ? kC : from + p.window, p.Lq - q0);
#pragma unroll
                        for (int i = 0; i < kC; ++i)
                            if (i < from || i >= until) pv[i] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) pk_p[i] = pack2<BF16>(pv[2 * i], pv[2 * i + 1]);
                    // Phase 2: dS^T = P^T o (dP^T - Delta).
                    ok = wait_bounded(&bar_of[os], oph, abort_v, p.timeout_ns) &&
                         wait_bounded(&bar_df, (uint32_t)uu & 1u, abort_v, p.timeout_ns);
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (ok) {
                    tc_fence_after_sync();
                    constexpr int kLd = kC >= 64 ? 32 : 16;  // dP^T columns per load (registers)
#pragma unroll
                    for (int h = 0; h < kC / kLd; ++h) {
                        uint32_t r[kLd];
                        tmem_ld<kLd>(tmem + lane_off + C::kTmDPT + c0 + h * kLd, r);
#pragma unroll
                        for (int i = 0; i < kLd; i += 4) {  // P o (dP - Delta), two per instruction
                            const float4 d = lds_f32x4(dlt_addr + (h * kLd + i) * 4);
                            float* q = pv + h * kLd + i;
                            f2_split(f2_mul(f2_make(q[0], q[1]),
                                            f2_sub(f2_make(__uint_as_float(r[i]),
                                                           __uint_as_float(r[i + 1])),
                                                   f2_make(d.x, d.y))),
                                     q[0], q[1]);
                            f2_split(f2_mul(f2_make(q[2], q[3]),
                                            f2_sub(f2_make(__uint_as_float(r[i + 2]),
                                                           __uint_as_float(r[i + 3])),
                                                   f2_make(d.z, d.w))),
                                     q[2], q[3]);
                        }
                    }
                }
                // Every slice of the quadrant has read its dP^T columns before any is
                // overwritten.  (All warps reach this barrier once per query tile on every path.)
                ok = bar_and(grp_bar, kGrpThreads, ok);
                if (!ok) break;
                {
                    tmem_st<kC / 2>(tmem + lane_off + C::kTmDPT + part * (kC / 2), pk_p);
                    uint32_t pk[kC / 2];
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) pk[i] = pack2<BF16>(pv[2 * i], pv[2 * i + 1]);
                    tmem_st<kC / 2>(tmem + lane_off + C::kTmDPT + 64 + part * (kC / 2), pk);
                }
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(&bar_ppd);
            }
            if (!ok) break;
            asm volatile("" : "+r"(id));  // (decoded anew: nothing of the item lives through the loop)
            DkdvItem it;
            dkdv_item(p, id, it);
            const int key0 = key - lane;
            const size_t coff = (size_t)part * C::kOutCols * 2;
            const int bhk = it.b * p.Hk + it.hk;
            uint8_t* dv0 = reinterpret_cast<uint8_t*>(p.dv) + row_offset(p.sdv, bhk, p.Hk, key0) + coff;
            uint8_t* dk0 = reinterpret_cast<uint8_t*>(p.dk) + row_offset(p.sdk, bhk, p.Hk, key0) + coff;
            if (empty) {
                if (it.part < 0 && key < p.Lk) {  // a row per lane: rare
#pragma unroll
                    for (int c = 0; c < C::kOutCols / 8; ++c) {
                        reinterpret_cast<uint4*>(dv0 + (size_t)lane * p.sdv.l * 2)[c] = make_uint4(0, 0, 0, 0);
                        reinterpret_cast<uint4*>(dk0 + (size_t)lane * p.sdk.l * 2)[c] = make_uint4(0, 0, 0, 0);
                    }
                }
                continue;
            }
            ok = wait_bounded(&bar_done, done_par, abort_v, p.timeout_ns);
            done_par ^= 1u;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            // tcgen05.ld waits for its data: the read-out is complete before this warp publishes
            // P^T / dS^T of the next item, which is what lets dK / dV of that item start.
            if (it.part >= 0) {
                part_out<C::kOutCols>(tmem + lane_off + C::kTmDK + part * C::kOutCols,
                                      p.part + (size_t)it.part * 2 * kTileRows * D, part, row);
                part_out<C::kOutCols>(tmem + lane_off + C::kTmDV + part * C::kOutCols,
                                      p.part + ((size_t)it.part * 2 + 1) * kTileRows * D, part, row);
            } else {
                // The warp's 32 key rows from key - lane, stored coalesced across the warp.
                tmem_rows_to_global_xpose<BF16, C::kOutCols>(
                    tmem + lane_off + C::kTmDV + part * C::kOutCols, dv0, (size_t)p.sdv.l * 2u, p.Lk - key0,
                    1.0f, lane);
                tmem_rows_to_global_xpose<BF16, C::kOutCols>(
                    tmem + lane_off + C::kTmDK + part * C::kOutCols, dk0, (size_t)p.sdk.l * 2u, p.Lk - key0,
                    p.scale, lane);
            }
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
struct DqCfg {
    static constexpr int kChunks = D / kChunkElems;
    static constexpr int kTileBytes = kTileRows * D * 2;
    static constexpr int kStages = (D == 128) ? 3 : 6;  // K/V ring depth
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kSmemBytes = kOffV + kStages * kTileBytes + 1024;
    // Elementwise warps per TMEM lane quadrant: at D = 64 the tensor core spends half as long
    // per key tile, so the elementwise phase is split over twice as many warps.
    static constexpr int kSplit = (D == 64) ? 4 : 2;
    static constexpr int kEwWarps = 4 * kSplit;
    static constexpr int kEwThreads = kEwWarps * 32;
    static constexpr int kProducerWarp = kEwWarps;
    static constexpr int kMmaWarp = kEwWarps + 1;
    static constexpr int kThreads = (kEwWarps + 2) * 32;
    static constexpr int kCols = 128 / kSplit;   // key columns per elementwise warp
    static constexpr int kOutCols = D / kSplit;  // dQ columns per elementwise warp
    static constexpr int kStageCols = D / 2 / kSplit;  // packed dO columns each warp stages
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kTmS = 0, kTmDP = 128, kTmDQ = 256;
    // dS has its own 64 columns, so dP_{j+1} never waits for dQ_j to have read dS_j.
    static constexpr uint32_t kTmDO = 256 + D;
    static constexpr uint32_t kTmDS = kTmDO + D / 2;
    static_assert(kTmDS + 64 <= kTmemCols, "TMEM budget");
    static constexpr uint32_t kIdescS = idesc_f16(BF16, 128, 128, false, false);
    static constexpr uint32_t kIdescG = idesc_f16(BF16, 128, D, false, true);
};

// dQ.
//
// DELTA: the same tiles' Delta = rowsum(P o dP) instead, summed in fp32, for the first p.delta_tiles query tiles that
// see a key.  The preprocess takes Delta from the rounded O, off by O's rounding and that of P in it; a row of few
// keys passes that on to all of its dS (error of dQ and dK relative to their rounding to 16 bits alone: 1.75 for a
// window of 8, 1.5 for 1024, whose first rows are the largest; with Delta from P and dP 1.45, dS's own rounding).
// Its price: 8 to 26 us where only the first 256 rows of a head see so few keys (8 x 4096, 32 heads of 128, window 1024:
// 26 of 1580 us); with window and first tokens below kDeltaKeys every query tile takes it, a quarter of the backward:
// windows of 16, 64, 128, 255 295, 294, 276, 292 of 1120, 1114, 1072, 1192 us (heads of 64: 200, 192, 184, 219 of 834,
// 818, 804, 947), where 256 takes 26 of 920 (20 of 742).
template <int D, bool BF16, bool DELTA>
__global__ void __launch_bounds__(DqCfg<D, BF16>::kThreads, 1)
    fa_window_dq_kernel(const __grid_constant__ WindowBwdParams p) {
    using C = DqCfg<D, BF16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    // Per key-tile iteration (phase = running iteration count over all tiles of this CTA):
    __shared__ uint64_t bar_sf, bar_df;     // S / dP complete
    __shared__ uint64_t bar_sr, bar_dpr;    // S / dP read: their columns may be overwritten
    __shared__ uint64_t bar_pd;             // dS written
    __shared__ uint64_t bar_dqd;            // dQ += dS K done: the dS columns may be overwritten
    __shared__ uint64_t bar_kvf[C::kStages], bar_kve[C::kStages];  // K/V ring full / empty
    // Per query tile (phase = tile count of this CTA):
    __shared__ uint64_t bar_q;    // Q_i landed in shared memory
    __shared__ uint64_t bar_qe;   // every S of the tile complete: the Q buffer may be refilled
    __shared__ uint64_t bar_qt;   // dO_i staged into TMEM
    __shared__ uint64_t bar_done; // every MMA of the tile complete: dQ_i final
    __shared__ uint64_t bar_dqr;  // dQ_i read out: the accumulator may be overwritten
    __shared__ uint64_t bar_fin;
    __shared__ WorkQueue queue;  // this CTA's query tiles, fetched from the pass's counter
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    volatile int* abort_v = &abort_flag;
    // Work ids: heads in L2-sized groups, the last query tiles first; the first q_first ones see no key.
    const int rows = DELTA ? p.delta_tiles : p.n_qtiles - p.q_first, total = rows * p.B * p.Hq;
    int* counter = p.sched + (DELTA ? 2 : 1);
    struct Tile {
        int bh, b, h, hk, qt, n_kv;
        KeyTiles keys;
    };
    auto tile_from = [&](int id, Tile& t) {
        int rank;
        tile_coords(id, p.B * p.Hq, rows, p.sched_group_q, t.bh, rank);
        t.b = t.bh / p.Hq;
        t.h = t.bh - t.b * p.Hq;
        t.hk = t.h / (p.Hq / p.Hk);
        t.qt = DELTA ? p.q_first + rank : p.n_qtiles - 1 - rank;
        const int first = t.qt * kTileRows, off = p.Lk - p.Lq;
        t.keys = key_tiles(first + off, imin(first + kTileRows, p.Lq) - 1 + off, p.window, p.sinks);
        t.n_kv = t.keys.count();
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar_kvf[s], 1);
            mbar_init(&bar_kve[s], 1);
        }
        mbar_init(&bar_sf, 1);
        mbar_init(&bar_df, 1);
        mbar_init(&bar_sr, C::kEwThreads);
        mbar_init(&bar_dpr, C::kEwThreads);
        mbar_init(&bar_pd, C::kEwThreads);
        mbar_init(&bar_dqd, 1);
        mbar_init(&bar_q, 1);
        mbar_init(&bar_qe, 1);
        mbar_init(&bar_qt, C::kEwThreads);
        mbar_init(&bar_done, 1);
        mbar_init(&bar_dqr, C::kEwThreads);
        mbar_init(&bar_fin, 1);
        queue_init(queue, 1 + C::kEwWarps);  // read by the MMA warp and the elementwise warps
        mbar_fence_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&tmem_base_sh, C::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base_sh;

    if (warp == C::kProducerWarp) {
        // ------------------------------ TMA producer ------------------------------
        // Fetches the tile ids (one round ahead).  Per tile: Q_i (once the previous tile's S
        // contractions have completed), then its K_j / V_j into the ring, which runs on across
        // tiles, so the next tile's first key tiles are already in flight while this one
        // finishes.
        if (lane == 0) {
            tma_prefetch_desc(&p.tm_k);
            tma_prefetch_desc(&p.tm_v);
            tma_prefetch_desc(&p.tm_q);
            bool ok = true;
            int gk = 0;       // K/V fills handed to the TMA unit
            int q_loads = 0;  // Q fills handed to the TMA unit
            Tile t;
            int next_id = queue_push(queue, 0, counter, total, false, abort_v, p.timeout_ns);
            for (int round = 0; ok; ++round) {
                const int id = next_id;
                if (id == -2) ok = false;
                if (id < 0) break;
                next_id = queue_push(queue, round + 1, counter, total, false, abort_v,
                                     p.timeout_ns);
                tile_from(id, t);
                if (q_loads > 0 &&
                    !wait_bounded(&bar_qe, (uint32_t)(q_loads - 1) & 1u, abort_v, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&bar_q, C::kTileBytes);
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load_4d(smem + C::kOffQ + c * kChunkBytes, &p.tm_q, &bar_q,
                                c * kChunkElems, t.qt * kTileRows, t.h, t.b);
                ++q_loads;
                for (int j = 0; j < t.n_kv; ++j) {
                    const int st = gk % C::kStages;
                    const uint32_t ph = (uint32_t)(gk / C::kStages) & 1u;
                    if (gk >= C::kStages &&
                        !wait_bounded(&bar_kve[st], ph ^ 1u, abort_v, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bar_kvf[st], 2 * C::kTileBytes);
                    const int key0 = t.keys.tile(j) * kTileRows;
                    for (int c = 0; c < C::kChunks; ++c) {
                        tma_load_4d(smem + C::kOffK + st * C::kTileBytes + c * kChunkBytes,
                                    &p.tm_k, &bar_kvf[st], c * kChunkElems, key0, t.hk, t.b);
                        tma_load_4d(smem + C::kOffV + st * C::kTileBytes + c * kChunkBytes,
                                    &p.tm_v, &bar_kvf[st], c * kChunkElems, key0, t.hk, t.b);
                    }
                    ++gk;
                }
            }
            if (!ok) record_timeout(p.status, abort_v);
            // Drain: no copy may still be landing when the CTA exits.
            if (q_loads > 0)
                wait_bounded(&bar_q, (uint32_t)(q_loads - 1) & 1u, nullptr, p.timeout_ns);
            for (int g = gk - 1; g >= 0 && g >= gk - C::kStages; --g)
                wait_bounded(&bar_kvf[g % C::kStages], (uint32_t)(g / C::kStages) & 1u, nullptr,
                             p.timeout_ns);
        }
    } else if (warp == C::kMmaWarp) {
        // ------------------------------ MMA issuer ------------------------------
        // The whole warp walks the loop (warp-uniform values); one elected lane issues.  g is
        // the running key-tile iteration over all of this CTA's tiles (ring slot and phase).
        auto k_base = [&](int g) {
            return smem_u32(smem + C::kOffK + (g % C::kStages) * C::kTileBytes);
        };
        auto v_base = [&](int g) {
            return smem_u32(smem + C::kOffV + (g % C::kStages) * C::kTileBytes);
        };
        auto wait_stage = [&](int g) {
            const bool r = wait_warp(&bar_kvf[g % C::kStages], (uint32_t)(g / C::kStages) & 1u,
                                     abort_v, p.timeout_ns);
            tc_fence_after_sync();
            return r;
        };
        auto issue_s = [&](int g) {  // S = Q K^T, both operands in shared memory
            const uint64_t kd = sdesc_kmajor_sw128(k_base(g));
            const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + C::kOffQ));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                mma_ss_w(tmem + C::kTmS, sdesc_advance(qd, off), sdesc_advance(kd, off),
                         C::kIdescS, kk > 0 ? 1u : 0u);
            }
            mma_commit_w(&bar_sf);
        };
        auto issue_dp = [&](int g) {  // dP = dO V^T, dO from TMEM
            const uint64_t vd = sdesc_kmajor_sw128(v_base(g));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
                mma_ts_w(tmem + C::kTmDP, tmem + C::kTmDO + kk * 8, sdesc_advance(vd, off),
                         C::kIdescS, kk > 0 ? 1u : 0u);
            }
            mma_commit_w(&bar_df);
        };
        bool ok = true;
        int g = 0;
        int tc = 0;
        Tile t;
        for (int round = 0; ok; ++round, ++tc) {
            const int id = queue_pop_warp(queue, round, abort_v, p.timeout_ns);
            if (id == -2) ok = false;
            if (id < 0) break;
            tile_from(id, t);
            const int n = t.n_kv;
            // Q_i landed and dO_i staged; the previous tile's last S and dP have been read (their
            // columns are reused); K_0 / V_0 of this tile landed.
            ok = wait_warp(&bar_q, (uint32_t)tc & 1u, abort_v, p.timeout_ns) &&
                 wait_warp(&bar_qt, (uint32_t)tc & 1u, abort_v, p.timeout_ns);
            if (ok && g > 0)
                ok = wait_warp(&bar_sr, (uint32_t)(g - 1) & 1u, abort_v, p.timeout_ns) &&
                     wait_warp(&bar_dpr, (uint32_t)(g - 1) & 1u, abort_v, p.timeout_ns);
            if (ok) ok = wait_stage(g);
            if (!ok) break;
            issue_s(g);
            if (n == 1) mma_commit_w(&bar_qe);  // the tile's only S: Q free once it completes
            issue_dp(g);
            if constexpr (DELTA) mma_commit_w(&bar_kve[g % C::kStages]);  // K_0, V_0 read
            for (int j = 0; j < n; ++j) {
                const int gg = g + j;
                const uint32_t par = (uint32_t)gg & 1u;
                if (j + 1 < n) {
                    // S of the next key tile as soon as this one's S has been read.
                    if (!wait_stage(gg + 1) || !wait_warp(&bar_sr, par, abort_v, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    issue_s(gg + 1);
                    if (j + 2 == n) mma_commit_w(&bar_qe);  // the tile's last S issued
                    // dP_{j+1} as soon as dP_j has been read (dS has its own columns).
                    if (!wait_warp(&bar_dpr, par, abort_v, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    issue_dp(gg + 1);
                    if constexpr (DELTA) mma_commit_w(&bar_kve[(gg + 1) % C::kStages]);
                }
                if constexpr (DELTA) continue;
                if (!wait_warp(&bar_pd, par, abort_v, p.timeout_ns) ||
                    (j == 0 && tc > 0 &&
                     !wait_warp(&bar_dqr, (uint32_t)(tc - 1) & 1u, abort_v, p.timeout_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint64_t kmd = sdesc_mnmajor_sw128(k_base(gg), kChunkBytes);
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk)
                    mma_ts_w(tmem + C::kTmDQ, tmem + C::kTmDS + kk * 8,
                             sdesc_advance(kmd, kk * 2048), C::kIdescG,
                             (j > 0 || kk > 0) ? 1u : 0u);
                mma_commit_w(&bar_kve[gg % C::kStages]);  // K_j, V_j fully read
                mma_commit_w(&bar_dqd);                   // dS_j consumed
            }
            if (!ok) break;
            if constexpr (!DELTA) mma_commit_w(&bar_done);
            g += n;
        }
        if (!ok && lane == 0) record_timeout(p.status, abort_v);
        mma_commit_w(&bar_fin);
        wait_warp(&bar_fin, 0, nullptr, p.timeout_ns);
    } else {
        // ------------------------------ elementwise warps ------------------------------
        constexpr int kC = C::kCols;
        const int quad = warp & 3;              // TMEM lane quadrant (query rows)
        const int part = warp >> 2;             // which kC key columns
        const int row = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const int c0 = part * kC;
        // Stage this warp's slice (D/kSplit elements) of tile t's dO row into TMEM as packed
        // 16-bit pairs (rows past L are zeros), and read the row's -LSE*log2(e) and Delta.
        auto stage_do = [&](const Tile& t, float& nl, float& dl) {
            constexpr int kE = D / C::kSplit;       // elements per warp slice
            constexpr int kW = C::kStageCols;       // packed 32-bit columns per slice
            const int q_row = t.qt * kTileRows + row;  // < Lqpad always
            const bool valid = q_row < p.Lq;
            const uint4* src = reinterpret_cast<const uint4*>(
                reinterpret_cast<const uint8_t*>(p.dout) + row_offset(p.sdo, t.bh, p.Hq, q_row) +
                (size_t)part * kE * 2);
            uint32_t w[kW];
#pragma unroll
            for (int v = 0; v < kW / 4; ++v) {
                const uint4 x = valid ? src[v] : make_uint4(0u, 0u, 0u, 0u);
                w[4 * v + 0] = x.x;
                w[4 * v + 1] = x.y;
                w[4 * v + 2] = x.z;
                w[4 * v + 3] = x.w;
            }
            nl = p.nlse2_pad[(size_t)t.bh * p.Lqpad + q_row];
            dl = p.delta_pad[(size_t)t.bh * p.Lqpad + q_row];
            tmem_st<kW>(tmem + lane_off + C::kTmDO + part * kW, w);
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(&bar_qt);
        };
        Tile cur, nxt;
        float nlse2 = 0.0f, dlt = 0.0f;  // -LSE * log2(e) and Delta of this thread's row
        const int id0 = queue_pop_warp(queue, 0, abort_v, p.timeout_ns);
        bool ok = id0 != -2;
        if constexpr (DELTA) ok = bar_and(1 + quad, 32 * C::kSplit, ok);
        const bool any = id0 >= 0;  // a CTA that starts late may find no tile left
        if (any) {
            tile_from(id0, cur);
            stage_do(cur, nlse2, dlt);
        }
        int g = 0;
        for (int round = 0, tc = 0; ok && any; ++round, ++tc) {
            const int idn = queue_pop_warp(queue, round + 1, abort_v, p.timeout_ns);
            if (idn == -2) {
                ok = false;
                if constexpr (!DELTA) break;  // (DELTA: the quadrant's warps meet below on every path)
            }
            const bool has_next = idn >= 0;
            if (has_next) tile_from(idn, nxt);
            const int n = cur.n_kv;
            const int q_row = cur.qt * kTileRows + row;
            const int pos = q_row + (p.Lk - p.Lq);
            const uint64_t dlt2 = f2_make(dlt, dlt);
            float nlse2_n = 0.0f, dlt_n = 0.0f;
            uint64_t sum2 = 0ull;  // DELTA: (+0.0f, +0.0f)
            for (int j = 0; ok && j < n; ++j) {
                const int gg = g + j;
                const int key0 = cur.keys.tile(j) * kTileRows + c0;
                const bool masked = hides_later(key0, kC, pos - lane) ||
                                    hides_earlier(key0, kC, pos - lane + 31, p.window, p.sinks);
                const uint32_t par = (uint32_t)gg & 1u;
                float pv[kC];
                ok = wait_bounded(&bar_sf, par, abort_v, p.timeout_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    tc_fence_after_sync();
                    uint32_t r[kC];
                    tmem_ld_cols<kC>(tmem + lane_off + C::kTmS + c0, r);
                    tc_fence_before_sync();
                    mbar_arrive(&bar_sr);
                    const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
                    const uint64_t shift2 = f2_make(nlse2, nlse2);
#pragma unroll
                    for (int i = 0; i < kC; i += 2) {  // two columns per f32x2 instruction
                        float y0, y1;
                        f2_split(f2_fma(f2_make(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                        scale2, shift2),
                                 y0, y1);
                        pv[i] = ex2_approx(y0);
                        pv[i + 1] = ex2_approx(y1);
                    }
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < kC; ++i)
                            if (i > pos - key0 || (i <= pos - p.window - key0 && i >= p.sinks - key0))
                                pv[i] = 0.0f;
                    }
                    ok = wait_bounded(&bar_df, par, abort_v, p.timeout_ns);
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (ok) {
                    tc_fence_after_sync();
                    constexpr int kLd = kC >= 64 ? 32 : 16;  // dP columns per load (registers)
#pragma unroll
                    for (int h = 0; h < kC / kLd; ++h) {
                        uint32_t r[kLd];
                        tmem_ld<kLd>(tmem + lane_off + C::kTmDP + c0 + h * kLd, r);
#pragma unroll
                        for (int i = 0; i < kLd; i += 2) {  // P o (dP - Delta), two at a time
                            float* q = pv + h * kLd + i;
                            const uint64_t dp = f2_make(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                            if constexpr (DELTA) sum2 = f2_fma(f2_make(q[0], q[1]), dp, sum2);
                            else f2_split(f2_mul(f2_make(q[0], q[1]), f2_sub(dp, dlt2)), q[0], q[1]);
                        }
                    }
                    tc_fence_before_sync();
                    mbar_arrive(&bar_dpr);  // this thread's dP columns are read
                }
                if (!ok) break;
                // dS has its own columns: wait until the previous dQ contraction (of this tile
                // or the last one of the previous tile) has read them.
                if (!DELTA && gg > 0) {
                    ok = wait_bounded(&bar_dqd, par ^ 1u, abort_v, p.timeout_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                if constexpr (!DELTA) {
                    uint32_t pk[kC / 2];
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) pk[i] = pack2<BF16>(pv[2 * i], pv[2 * i + 1]);
                    tmem_st<kC / 2>(tmem + lane_off + C::kTmDS + part * (kC / 2), pk);
                    tmem_st_wait();
                    tc_fence_before_sync();
                    mbar_arrive(&bar_pd);
                }
                // The tile's last dP has completed (it was read above), so the next tile's dO
                // may take the dO columns now: the MMA warp can start that tile's dP while
                // this tile's dQ is read out.
                if (j == n - 1 && has_next) stage_do(nxt, nlse2_n, dlt_n);
            }
            if constexpr (DELTA) {
                // The quadrant's warps add up by way of TMEM columns that are free here (of dS and of dQ, tile
                // after tile: at this barrier the sums of two tiles ago have been read).
                const uint32_t at = tmem + lane_off + ((tc & 1) ? C::kTmDQ : C::kTmDS);
                float lo, hi;
                f2_split(sum2, lo, hi);
                uint32_t mine[8] = {__float_as_uint(lo + hi), 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                tmem_st8(at + 8 * part, mine);
                tmem_st_wait();
                tc_fence_before_sync();
                ok = bar_and(1 + quad, 32 * C::kSplit, ok);
                if (!ok) break;
                tc_fence_after_sync();
                if (part == 0) {
                    uint32_t all[8 * C::kSplit];
                    tmem_ld<8 * C::kSplit>(at, all);
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < C::kSplit; ++i) sum += __uint_as_float(all[8 * i]);
                    p.delta_pad[(size_t)cur.bh * p.Lqpad + q_row] = sum;
                    tc_fence_before_sync();
                }
            } else {
                if (ok) {
                    ok = wait_bounded(&bar_done, (uint32_t)tc & 1u, abort_v, p.timeout_ns);
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (!ok) break;
                tc_fence_after_sync();
                uint8_t* dst_row = reinterpret_cast<uint8_t*>(p.dq) +
                                   row_offset(p.sdq, cur.bh, p.Hq, q_row) + part * C::kOutCols * 2;
                tmem_row_to_global<BF16, C::kOutCols>(tmem + lane_off + C::kTmDQ + part * C::kOutCols,
                                                      dst_row, p.scale, q_row < p.Lq);
                tc_fence_before_sync();
                mbar_arrive(&bar_dqr);  // the accumulator is read: the next tile may overwrite it
            }
            g += n;
            if (!has_next) break;
            cur = nxt;
            nlse2 = nlse2_n;
            dlt = dlt_n;
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

// Sums the fp32 parts of the first tokens' key tiles in their order: one thread per row and eight columns.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa_window_join_kernel(const WindowBwdParams p) {
    const int tile = blockIdx.x;  // (batch and key head) * split_tiles + key tile
    const int bhk = tile / p.split_tiles, kt = tile - bhk * p.split_tiles;
    const QueryTiles q = query_tiles(kt, p.Lq, p.Lk - p.Lq, p.window, p.sinks);
    const int units = (q.hi - q.lo) * (p.Hq / p.Hk);
    const int e = blockIdx.y * 256 + threadIdx.x;  // of 2 * (D / 8) * 128
    const int row = e & (kTileRows - 1), c = (e >> 7) % (D / 8), which = (e >> 7) / (D / 8);
    const int key = kt * kTileRows + row;
    if (key >= p.Lk) return;
    float x[8] = {};
    for (int i = 0; i < p.parts; ++i) {
        if (part_start(units, i, p.parts) == part_start(units, i + 1, p.parts)) continue;  // nobody wrote it
        const float4* src = reinterpret_cast<const float4*>(
                                p.part + (((size_t)tile * p.parts + i) * 2 + which) * kTileRows * D) +
                            (size_t)2 * c * kTileRows + row;
        const float4 a = src[0], b = src[kTileRows];
        x[0] += a.x;
        x[1] += a.y;
        x[2] += a.z;
        x[3] += a.w;
        x[4] += b.x;
        x[5] += b.y;
        x[6] += b.z;
        x[7] += b.w;
    }
    const float m = which ? 1.0f : p.scale;
    uint8_t* dst = which ? reinterpret_cast<uint8_t*>(p.dv) + row_offset(p.sdv, bhk, p.Hk, key)
                         : reinterpret_cast<uint8_t*>(p.dk) + row_offset(p.sdk, bhk, p.Hk, key);
    reinterpret_cast<uint4*>(dst)[c] = make_uint4(pack2<BF16>(x[0] * m, x[1] * m), pack2<BF16>(x[2] * m, x[3] * m),
                                                  pack2<BF16>(x[4] * m, x[5] * m), pack2<BF16>(x[6] * m, x[7] * m));
}

template <int D, bool BF16>
cudaError_t launch_dkdv_t(const WindowBwdParams& p, cudaStream_t s) {
    using C = DkdvCfg<D, BF16>;
    constexpr int kSmem = C::kOffBar + (int)sizeof(DkdvBarsT<D, BF16>);
    static_assert(kSmem <= 232448, "dynamic shared memory over the 227 KB per-block limit");
    constexpr auto kern = fa_window_dkdv_kernel<D, BF16>;
    const cudaError_t e = allow_shared_once<kern>(kSmem);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    const int grid = sms > 0 && sms < p.dkdv_items ? sms : p.dkdv_items;
    return launch_kernel(kern, (unsigned)grid, C::kThreads, kSmem, s, p);
}

template <int D, bool BF16, bool DELTA>
cudaError_t launch_dq_t(const WindowBwdParams& p, cudaStream_t s) {
    using C = DqCfg<D, BF16>;
    constexpr auto kern = fa_window_dq_kernel<D, BF16, DELTA>;
    const cudaError_t e = allow_shared_once<kern>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int total = (DELTA ? p.delta_tiles : p.n_qtiles - p.q_first) * p.B * p.Hq, sms = sm_count();
    const int grid = sms > 0 && sms < total ? sms : total;
    return launch_kernel(kern, (unsigned)grid, C::kThreads, C::kSmemBytes, s, p);
}

template <int D, bool BF16>
cudaError_t launch_join_t(const WindowBwdParams& p, cudaStream_t s) {
    return launch_kernel(fa_window_join_kernel<D, BF16>,
                         dim3((unsigned)(p.B * p.Hk * p.split_tiles), 2 * (D / 8) * kTileRows / 256), dim3(256), 0,
                         s, p);
}

}  // namespace

void window_bwd_plan(WindowBwdParams* p) {
    const int off = p->Lk - p->Lq, group = p->Hq / p->Hk, heads = p->B * p->Hk;
    const int n_sink = imin((p->sinks + kTileRows - 1) / kTileRows, p->n_ktiles);
    const int usual = group * imin((p->window + 254) / kTileRows, p->n_qtiles);
    const QueryTiles q0 = query_tiles(0, p->Lq, off, p->window, p->sinks);
    const int heavy = group * (q0.hi - q0.lo);
    // Half of an SM's share at most, but no less than a window's item.
    const long long all = (long long)heads * ((long long)n_sink * heavy + (long long)(p->n_ktiles - n_sink) * usual);
    const long long share = (all + 2 * kWindowSms - 1) / (2 * kWindowSms);
    const int most = (int)(share > usual ? share : usual);
    p->split_tiles = 2LL * heavy > 3LL * usual ? n_sink : 0;
    p->parts = p->split_tiles > 0 && 2LL * heavy > 3LL * most ? (heavy + most - 1) / most : 1;
    // Query tiles in which some row sees fewer than kDeltaKeys keys: all of them under a short window, else the first.
    const long long seen = (long long)p->window + imin(p->sinks, p->Lk - p->window);
    const int short_rows = seen < kDeltaKeys ? p->Lq : kDeltaKeys - off;  // rows in front of this one
    p->delta_tiles = imax(imin((short_rows + kTileRows - 1) / kTileRows, p->n_qtiles) - p->q_first, 0);
    p->dkdv_items = heads * (p->split_tiles * p->parts + p->n_ktiles - p->split_tiles);
}

cudaError_t launch_window_dkdv(const WindowBwdParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_dkdv_t<64, true>(p, s) : launch_dkdv_t<64, false>(p, s);
    return bf16 ? launch_dkdv_t<128, true>(p, s) : launch_dkdv_t<128, false>(p, s);
}
cudaError_t launch_window_dq(const WindowBwdParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_dq_t<64, true, false>(p, s) : launch_dq_t<64, false, false>(p, s);
    return bf16 ? launch_dq_t<128, true, false>(p, s) : launch_dq_t<128, false, false>(p, s);
}
cudaError_t launch_window_delta(const WindowBwdParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_dq_t<64, true, true>(p, s) : launch_dq_t<64, false, true>(p, s);
    return bf16 ? launch_dq_t<128, true, true>(p, s) : launch_dq_t<128, false, true>(p, s);
}
cudaError_t launch_window_join(const WindowBwdParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_join_t<64, true>(p, s) : launch_join_t<64, false>(p, s);
    return bf16 ? launch_join_t<128, true>(p, s) : launch_join_t<128, false>(p, s);
}

}  // namespace fa
