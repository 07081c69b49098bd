// fa_window.cu -- C entry points of attention under a sliding window with first tokens that stay
// visible: argument checks, tensor maps, launches.  The kernels are in fa_window_fwd.cu and
// fa_window_bwd.cu.
#include <cfloat>
#include <cmath>
#include <cstring>

#include "fa_host.h"
#include "fa_ptx.cuh"
#include "fa_window_sched.h"

using namespace fa;

namespace {

constexpr int kMaxLen = (1 << 30) - 1024;  // Lq + Lk and what a tile adds to them stay below 2^31

struct Shape {
    bool empty;  // no output row
    int n_qtiles, n_ktiles, Lqpad, window, sinks;
};

fa_status check_window(int B, int Hq, int Hk, int Lq, int Lk, int D, int window, int sinks, float scale,
                       int dtype, Shape* sh) {
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
    if (B < 0 || Hq < 0 || Hk < 0 || Lq < 0 || Lk < 0 || D <= 0) return FA_ERR_INVALID_ARG;
    if (window < 1 || sinks < 0 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    sh->empty = B == 0 || Hq == 0 || Lq == 0;
    if (B > 0 && Hq > 0 && (Hk == 0 || Hq % Hk != 0)) return FA_ERR_INVALID_ARG;
    if (Lq > kMaxLen || Lk > kMaxLen) return FA_ERR_UNSUPPORTED;
    sh->n_qtiles = (Lq + kTileRows - 1) / kTileRows;
    sh->n_ktiles = (Lk + kTileRows - 1) / kTileRows;
    sh->Lqpad = sh->n_qtiles * kTileRows;
    if ((long long)B * Hq > 0x7fffffffLL || (long long)B * Hq * sh->n_qtiles > 0x7fffffffLL ||
        (long long)B * Hk * sh->n_ktiles > 0x7fffffffLL - (1 << 20))
        return FA_ERR_UNSUPPORTED;
    sh->window = imin(window, imax(Lk, 1));  // (a larger one sees no more)
    sh->sinks = imin(sinks, Lk);
    return FA_OK;
}

// [B, H, L, D] with element strides as 4-D {D, L, H, B}, boxes of 64 elements x 128 rows; rows past L
// read as zeros.
bool make_rows_map(CUtensorMap* m, const void* ptr, int B, int H, int L, int D, const Strides& st, bool bf16) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)L, (cuuint64_t)H, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)st.l * 2, (cuuint64_t)st.h * 2, (cuuint64_t)st.b * 2};
    const cuuint32_t box[4] = {(cuuint32_t)kChunkElems, (cuuint32_t)kTileRows, 1, 1};
    return make_tiled_map(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ptr, 4,
                          dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Key heads per schedule group (tile_coords).  The items that run at the same time, one per SM, are some
// consecutive tiles of every head of a group; what they stream is `span` rows of a head and one more tile of
// them for each further tile, `row_bytes` each.  As many heads as keep that within kStreamed of L2.
constexpr long long kStreamed = 48LL << 20;
int sched_group(long long row_bytes, int span, int len, int items_per_tile, int heads) {
    for (int g = heads; g > 1; g = g > 2 * kWindowSms ? g / 2 : g - 1) {
        const int at_once = imin(g, kWindowSms), tiles = kWindowSms / (g * items_per_tile);
        const long long rows = imin(len, span + kTileRows * (tiles < 1 ? 1 : tiles));
        if (at_once * rows * row_bytes <= kStreamed) return g;
    }
    return 1;
}

// The plan of the backward pass and its workspace: the two vectors, the parts, the counters.
size_t bwd_plan(const Shape& sh, int B, int Hq, int Hk, int Lq, int Lk, int D, WindowBwdParams* p,
                size_t* part_at, size_t* sched_at) {
    std::memset(p, 0, sizeof(*p));
    p->B = B;
    p->Hq = Hq;
    p->Hk = Hk;
    p->Lq = Lq;
    p->Lk = Lk;
    p->Lqpad = sh.Lqpad;
    p->n_qtiles = sh.n_qtiles;
    p->n_ktiles = sh.n_ktiles;
    p->window = sh.window;
    p->sinks = sh.sinks;
    p->q_first = Lq > Lk ? (Lq - Lk) / kTileRows : 0;
    window_bwd_plan(p);
    *part_at = 2u * (size_t)B * Hq * sh.Lqpad * 4u;
    *sched_at = *part_at +
                (p->parts > 1 ? (size_t)B * Hk * p->split_tiles * p->parts * 2u * kTileRows * D * 4u : 0u);
    return *sched_at + kSchedBytes;
}

}  // namespace

extern "C" {

fa_status fa_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                        const fa_strides* strides, int B, int Hq, int Hk, int Lq, int Lk, int D, int window,
                        int sinks, float scale, int dtype, void* stream) {
    TraceDisarm disarm;
    Shape sh;
    const fa_status st = check_window(B, Hq, Hk, Lq, Lk, D, window, sinks, scale, dtype, &sh);
    if (st != FA_OK) return st;
    if (sh.empty) return FA_OK;
    if (Lk == 0) return FA_ERR_UNSUPPORTED;  // queries but no key at all
    if (!q || !k || !v || !o || !lse || !strides) return FA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, (const void*)o, (const void*)lse})
        if (!aligned16(ptr)) return FA_ERR_INVALID_ARG;
    Strides sq, sk, sv, so;
    if (!take_strides(strides[0], B, Hq, &sq) || !take_strides(strides[1], B, Hk, &sk) ||
        !take_strides(strides[2], B, Hk, &sv) || !take_strides(strides[3], B, Hq, &so))
        return FA_ERR_INVALID_ARG;
    const Range ro = extent(o, so, B, Hq, Lq, D), rl = range(lse, (size_t)B * Hq * Lq * 4u);
    const void* in[3] = {q, k, v};
    const Strides in_st[3] = {sq, sk, sv};
    for (int i = 0; i < 3; ++i) {
        const int H = i ? Hk : Hq, L = i ? Lk : Lq;
        const Range r = extent(in[i], in_st[i], B, H, L, D);
        if (overlap(rl, r)) return FA_ERR_INVALID_ARG;
        // o may be another part of one packed tensor.
        if (overlap(ro, r) && !(L == Lq && packed_parts(o, so, Hq, in[i], in_st[i], H, B, L, D)))
            return FA_ERR_INVALID_ARG;
    }
    if (overlap(ro, rl)) return FA_ERR_INVALID_ARG;

    WindowFwdParams p;
    std::memset(&p, 0, sizeof(p));
    const bool bf16 = dtype == FA_BF16;
    if (!bind_context()) return FA_ERR_CUDA;
    if (!make_rows_map(&p.tm_q, q, B, Hq, Lq, D, sq, bf16) || !make_rows_map(&p.tm_k, k, B, Hk, Lk, D, sk, bf16) ||
        !make_rows_map(&p.tm_v, v, B, Hk, Lk, D, sv, bf16))
        return FA_ERR_CUDA;
    p.o = o;
    p.so = so;
    p.lse = lse;
    p.Lq = Lq;
    p.Lk = Lk;
    p.Hq = Hq;
    p.Hk = Hk;
    p.B = B;
    p.window = sh.window;
    p.sinks = sh.sinks;
    p.single = (long long)B * Hq * sh.n_qtiles <= kWindowSms;
    p.head_pairs = !p.single && (Hq / Hk) % 2 == 0;
    p.columns = p.head_pairs ? B * (Hq / 2) : B * Hq;
    p.rows = p.head_pairs || p.single ? sh.n_qtiles : (sh.n_qtiles + 1) / 2;
    const int per_key_head = p.columns / (B * Hk);
    const int span = imin(Lk, sh.window + sh.sinks + kTileRows);
    p.sched_group = per_key_head * sched_group(4 * D, span, Lk, per_key_head, B * Hk);
    // (The softmax takes the maximum of the stored scores: a negative scale is moved into the
    // contraction as an exact sign flip, and the multiplier keeps a masked -inf at -inf.)
    p.scale_log2 = std::fmax(std::fabs(scale) * 1.4426950408889634f, FLT_MIN);
    p.s_negate = scale < 0.0f ? kIdescNegateA : 0u;
    p.status = status_ptr();
    p.timeout_ns = wait_timeout_ns();
    if (!p.status) return FA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (traced_launch(0, s, [&] { return launch_window_fwd(p, D, bf16, s); }) != cudaSuccess) return FA_ERR_CUDA;
    if (Lq > Lk) {  // the first Lq - Lk rows see no key
        FwdParams e;
        std::memset(&e, 0, sizeof(e));
        e.o = o;
        e.so = so;
        e.lse = lse;
        e.Lq = Lq;
        e.H = Hq;
        e.BH = B * Hq;
        if (traced_launch(1, s, [&] { return launch_fwd_empty_rows(e, D, Lq - Lk, s); }) != cudaSuccess)
            return FA_ERR_CUDA;
    }
    return FA_OK;
}

size_t fa_window_bwd_workspace_bytes(int B, int Hq, int Hk, int Lq, int Lk, int D, int window, int sinks) {
    Shape sh;
    if (check_window(B, Hq, Hk, Lq, Lk, D, window, sinks, 1.0f, FA_BF16, &sh) != FA_OK || sh.empty || Lk == 0)
        return 0;
    WindowBwdParams p;
    size_t part_at, sched_at;
    return bwd_plan(sh, B, Hq, Hk, Lq, Lk, D, &p, &part_at, &sched_at);
}

fa_status fa_window_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                        const fa_strides* strides, int B, int Hq, int Hk, int Lq, int Lk, int D, int window,
                        int sinks, float scale, int dtype, void* stream) {
    TraceDisarm disarm;
    Shape sh;
    const fa_status st = check_window(B, Hq, Hk, Lq, Lk, D, window, sinks, scale, dtype, &sh);
    if (st != FA_OK) return st;
    if (B == 0 || Hq == 0 || (Lq == 0 && Lk == 0)) return FA_OK;
    if (Lq == 0 || Lk == 0) return FA_ERR_UNSUPPORTED;
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace || !strides)
        return FA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, o, dout, (const void*)lse, (const void*)dq, (const void*)dk, (const void*)dv,
                            (const void*)workspace})
        if (!aligned16(ptr)) return FA_ERR_INVALID_ARG;
    WindowBwdParams p;
    size_t part_at, sched_at;
    const size_t need = bwd_plan(sh, B, Hq, Hk, Lq, Lk, D, &p, &part_at, &sched_at);
    if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
    const int heads[8] = {Hq, Hk, Hk, Hq, Hq, Hq, Hk, Hk}, len[8] = {Lq, Lk, Lk, Lq, Lq, Lq, Lk, Lk};
    const void* ptrs[8] = {q, k, v, o, dout, dq, dk, dv};
    Strides s8[8];
    Range r[10];
    for (int i = 0; i < 8; ++i) {
        if (!take_strides(strides[i], B, heads[i], &s8[i])) return FA_ERR_INVALID_ARG;
        r[i] = extent(ptrs[i], s8[i], B, heads[i], len[i], D);
    }
    r[8] = range(workspace, need);
    r[9] = range(lse, (size_t)B * Hq * Lq * 4u);
    for (int a = 5; a < 9; ++a) {
        if (overlap(r[a], r[9])) return FA_ERR_INVALID_ARG;
        for (int b = 0; b < a; ++b) {
            if (!overlap(r[a], r[b])) continue;
            // A gradient may be another part of one packed tensor.
            const bool packed = a < 8 && len[a] == len[b] &&
                                packed_parts(ptrs[a], s8[a], heads[a], ptrs[b], s8[b], heads[b], B, len[a], D);
            if (!packed) return FA_ERR_INVALID_ARG;
        }
    }
    const bool bf16 = dtype == FA_BF16;
    if (!bind_context()) return FA_ERR_CUDA;
    if (!make_rows_map(&p.tm_q, q, B, Hq, Lq, D, s8[0], bf16) ||
        !make_rows_map(&p.tm_k, k, B, Hk, Lk, D, s8[1], bf16) ||
        !make_rows_map(&p.tm_v, v, B, Hk, Lk, D, s8[2], bf16) ||
        !make_rows_map(&p.tm_do, dout, B, Hq, Lq, D, s8[4], bf16))
        return FA_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* nlse2 = reinterpret_cast<float*>(ws);
    float* delta = nlse2 + (size_t)B * Hq * sh.Lqpad;
    p.dout = dout;
    p.sdo = s8[4];
    p.nlse2_pad = nlse2;
    p.delta_pad = delta;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.sdq = s8[5];
    p.sdk = s8[6];
    p.sdv = s8[7];
    const int group = Hq / Hk, span = imin(Lk, sh.window + sh.sinks + kTileRows);
    p.sched_group_k = sched_group(4LL * D * group, sh.window + kTileRows, Lq, 1, B * Hk);
    p.sched_group_q = group * sched_group(4 * D, span, Lk, group, B * Hk);
    p.part = reinterpret_cast<float*>(ws + part_at);
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.sched = reinterpret_cast<int*>(ws + sched_at);
    p.status = status_ptr();
    p.timeout_ns = wait_timeout_ns();
    if (!p.status) return FA_ERR_CUDA;

    BwdPreParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.o = o;
    pp.dout = dout;
    pp.dq = dq;
    pp.so = s8[3];
    pp.sdo = s8[4];
    pp.sdq = s8[5];
    pp.lse = lse;
    pp.nlse2_pad = nlse2;
    pp.delta_pad = delta;
    pp.sched = p.sched;
    pp.Lq = Lq;
    pp.Lqpad = sh.Lqpad;
    pp.H = Hq;
    pp.BH = B * Hq;
    pp.D = D;
    pp.first_seen_row = Lq > Lk ? Lq - Lk : 0;  // rows in front of it see no key: dQ = 0
    pp.bf16 = bf16 ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int n = 0;
    if (traced_launch(n++, s, [&] { return launch_bwd_pre(pp, s); }) != cudaSuccess) return FA_ERR_CUDA;
    if (p.delta_tiles > 0 &&
        traced_launch(n++, s, [&] { return launch_window_delta(p, D, bf16, s); }) != cudaSuccess)
        return FA_ERR_CUDA;
    if (traced_launch(n++, s, [&] { return launch_window_dkdv(p, D, bf16, s); }) != cudaSuccess)
        return FA_ERR_CUDA;
    if (p.parts > 1 &&
        traced_launch(n++, s, [&] { return launch_window_join(p, D, bf16, s); }) != cudaSuccess)
        return FA_ERR_CUDA;
    return traced_launch(n++, s, [&] { return launch_window_dq(p, D, bf16, s); }) == cudaSuccess ? FA_OK
                                                                                                : FA_ERR_CUDA;
}

}  // extern "C"
