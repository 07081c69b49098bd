// fa_serve.cu -- C entry points of the operators around attention: rotary positions, the paged
// cache's writing and reading, the decode step with grouped heads and that with a shared prefix.
// Argument checks and launches; the kernels are in fa_rotary.cu, fa_cache.cu, fa_decode_gqa.cu and
// fa_prefix.cu.
#include <cfloat>
#include <cmath>
#include <cstring>

#include "fa_host.h"
#include "fa_overlap.h"

using namespace fa;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The same layout: equal strides of the dimensions that have more than one entry.
bool same(const Strides& a, const Strides& b, int B, int H, int L) {
    return (B <= 1 || a.b == b.b) && (H <= 1 || a.h == b.h) && (L <= 1 || a.l == b.l);
}
// Parts of one packed tensor: the same layout, extents that overlap, no element in common.
bool packed_parts(const void* a, const Strides& sa, int Ha, const void* b, const Strides& sb, int Hb, int B,
                  int L, int D) {
    const intptr_t pa = reinterpret_cast<intptr_t>(a), pb = reinterpret_cast<intptr_t>(b);
    if (!same(sa, sb, B, Ha < Hb ? Ha : Hb, L)) return false;
    const long long h = Ha > 1 ? sa.h : sb.h;
    return pa < pb ? interleave_apart((pb - pa) / 2, B, Ha, Hb, L, D, sa.b, h, sa.l)
                   : interleave_apart((pa - pb) / 2, B, Hb, Ha, L, D, sa.b, h, sa.l);
}

// The rotation of fa_rotary and fa_cache_append; freqs may be null only with rotary_dim = 0.
fa_status check_rotation(const int64_t* freqs, int rotary_dim, float mscale, int interleaved, int D,
                         RotaryParams* out) {
    if (rotary_dim < 0 || rotary_dim > D || (rotary_dim & 1)) return FA_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || !std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
    if (rotary_dim > 0 && (!freqs || !aligned8(freqs))) return FA_ERR_INVALID_ARG;
    out->freqs = reinterpret_cast<const long long*>(freqs);
    out->rotary_dim = rotary_dim;
    out->mscale = mscale;
    out->interleaved = interleaved;
    return FA_OK;
}

// Bytes of a paged cache's values and, for e4m3, of its exponents.
size_t cache_bytes(int num_pages, int H, int D, int cache_dtype) {
    return (size_t)num_pages * H * kPageTokens * D * (cache_dtype == FA_CACHE_E4M3 ? 1u : 2u);
}
size_t exp_bytes(int num_pages, int H) { return (size_t)num_pages * H * kPageTokens; }

// The kernels count rows up to the end of the last tile in 32 bits.
constexpr int kMaxTokens = 0x7fffffff - 1023;

// Sizes and flags shared by the calls on a paged cache.
fa_status check_cache(int B, int H, int L, int D, int num_pages, int max_pages, int dtype,
                      int cache_dtype) {
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
    if (cache_dtype != FA_CACHE_16BIT && cache_dtype != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
    if (B < 0 || H < 0 || L < 0 || D <= 0 || num_pages < 0 || max_pages < 0)
        return FA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535 || max_pages > 0x7fffffff / kPageTokens || L > kMaxTokens)
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// Pointers of a paged cache.
bool cache_pointers_ok(const void* kc, const void* vc, const void* ke, const void* ve,
                       const void* tables, const void* lens, int num_pages, int max_pages,
                       int cache_dtype) {
    if (num_pages > 0 && (!kc || !vc)) return false;
    if (num_pages > 0 && cache_dtype == FA_CACHE_E4M3 && (!ke || !ve)) return false;
    if (!lens || (max_pages > 0 && !tables)) return false;
    return aligned16(kc) && aligned16(vc) && aligned16(ke) && aligned16(ve) && aligned4(tables) &&
           aligned4(lens);
}

// Tensor map of a paged cache: one box is the 16 rows of a page's head (128 bytes of each at most).
bool make_cache_map(CUtensorMap* m, const void* cache, int num_pages, int H, int D, int dtype,
                    bool q8) {
    const cuuint64_t row = (cuuint64_t)D * (q8 ? 1 : 2);
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)kPageTokens, (cuuint64_t)num_pages * H};
    const cuuint64_t strides[2] = {row, row * kPageTokens};
    const cuuint32_t inner = row < 128 ? 64 : 128;  // bytes
    const cuuint32_t box[3] = {q8 ? inner : inner / 2, (cuuint32_t)kPageTokens, 1};
    return make_tiled_map(m,
                          q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                             : (dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16),
                          cache, 3, dims, strides, box,
                          inner == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Sizes of a decode step with grouped heads.
fa_status check_decode(int B, int Hq, int Hk, int D, int num_pages, int max_pages, float scale,
                       int dtype, int cache_dtype) {
    if (Hq < 0 || Hk < 0 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(B, Hk, 0, D, num_pages, max_pages, dtype, cache_dtype);
    if (st != FA_OK) return st;
    if (B == 0 || Hq == 0) return FA_OK;
    if (Hk == 0 || Hq % Hk != 0) return FA_ERR_INVALID_ARG;
    if ((long long)B * Hq > 0x7fffffffLL || (long long)num_pages * Hk > 0x7fffffffLL ||
        (long long)B * max_pages > 0x7fffffffLL || Hq > 65535)
        return FA_ERR_UNSUPPORTED;
    // A warp counts its pages in 32 bits (units of one query block at least 8 wide).
    if ((long long)B * max_pages * ((Hq + 7) / 8 + Hk) > 1LL << 40) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

int q_blocks_of(int group) { return (group + gqa_q_rows(group) - 1) / gqa_q_rows(group); }

int slot_rows_of(int group) { return group < gqa_q_rows(group) ? group : gqa_q_rows(group); }

// Workspace of a decode step, in bytes from its start.
struct DecodeWorkspace {
    size_t unit_parts, slot_o, slot_lse, full_o, full_lse, prefix_o, prefix_lse, bytes;
    int warps;
};
DecodeWorkspace decode_workspace(int B, int Hq, int Hk, int D, int max_pages, bool shared,
                                 int n_prefix) {
    DecodeWorkspace w;
    const int chunk = B < kGqaMaxSequences ? B : kGqaMaxSequences;
    w.warps = gqa_warps(chunk, Hk, Hq / Hk, max_pages);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 15) & ~(size_t)15;
        return here;
    };
    const size_t slots = 2 * (size_t)w.warps * gqa_rounds(chunk, Hk, Hq / Hk) * slot_rows_of(Hq / Hk);
    const size_t rows = (size_t)B * Hq;
    w.unit_parts = take((size_t)chunk * Hk * q_blocks_of(Hq / Hk) * 8);
    w.slot_o = take(slots * D * 4);
    w.slot_lse = take(slots * 4);
    w.full_o = take(shared ? rows * D * 4 : 0);
    w.full_lse = take(shared ? rows * 4 : 0);
    w.prefix_o = take(rows * n_prefix * D * 4);
    w.prefix_lse = take(rows * n_prefix * 4);
    w.bytes = at;
    return w;
}

// The decode kernel and the merge for the batch, kGqaMaxSequences at a time.  p holds everything
// but what depends on the workspace and the chunk; `kernel` counts the traced kernels so far.
cudaError_t run_decode(GqaParams p, int B, int D, bool bf16, bool q8, uint8_t* ws,
                       const DecodeWorkspace& w, int n_prefix, int busy_sms, int kernel, cudaStream_t s) {
    const size_t row_o = (size_t)p.Hq * D;
    p.q_blocks = q_blocks_of(p.group);
    p.slot_rows = slot_rows_of(p.group);
    p.unit_parts = reinterpret_cast<int2*>(ws + w.unit_parts);
    p.slot_o = reinterpret_cast<float*>(ws + w.slot_o);
    p.slot_lse = reinterpret_cast<float*>(ws + w.slot_lse);
    for (int b0 = 0; b0 < B; b0 += kGqaMaxSequences) {
        GqaParams c = p;
        c.B = B - b0 < kGqaMaxSequences ? B - b0 : kGqaMaxSequences;
        c.q = static_cast<const uint16_t*>(p.q) + b0 * row_o;
        c.o = static_cast<uint16_t*>(p.o) + b0 * row_o;
        c.lse = p.lse + (size_t)b0 * p.Hq;
        c.block_tables = p.block_tables ? p.block_tables + (size_t)b0 * p.max_pages : nullptr;
        c.seq_lens = p.seq_lens + b0;
        c.full_o = reinterpret_cast<float*>(ws + w.full_o) + b0 * row_o;
        c.full_lse = reinterpret_cast<float*>(ws + w.full_lse) + (size_t)b0 * p.Hq;
        c.early = p.early && b0 == 0;
        c.short_step = !p.parts_only && gqa_short(c.B, p.Hk, p.group, p.max_pages, D, q8);
        c.rounds = gqa_rounds(c.B, p.Hk, p.group);
        c.warps = gqa_launched_warps(c.B, p.Hk, p.group, p.max_pages, D, q8, c.early ? busy_sms : 0);
        cudaError_t e = traced_launch(kernel++, s, [&] { return launch_decode_gqa(c, D, bf16, q8, s); });
        if (e != cudaSuccess) return e;
        if (c.short_step) continue;  // (its clusters have joined their parts)
        MergeParams m;
        std::memset(&m, 0, sizeof(m));
        m.prefix_o = reinterpret_cast<float*>(ws + w.prefix_o) + b0 * row_o * n_prefix;
        m.prefix_lse = reinterpret_cast<float*>(ws + w.prefix_lse) + (size_t)b0 * p.Hq * n_prefix;
        m.n_prefix = n_prefix;
        m.slot_o = c.slot_o;
        m.slot_lse = c.slot_lse;
        m.full_o = c.full_o;
        m.full_lse = c.full_lse;
        m.unit_parts = c.unit_parts;
        m.o = c.o;
        m.lse = c.lse;
        m.rows = c.B * p.Hq;
        m.B = c.B;
        m.Hq = p.Hq;
        m.Hk = p.Hk;
        m.group = p.group;
        m.q_rows = gqa_q_rows(p.group);
        m.q_blocks = p.q_blocks;
        m.slot_rows = p.slot_rows;
        m.workers = c.warps * c.rounds;
        e = traced_launch(kernel++, s, [&] { return launch_merge(m, D, bf16, s); });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

extern "C" {

fa_status fa_rotary_freqs(int rotary_dim, double base, int scaling, double factor,
                          double original_len, int64_t* freqs, float* mscale) {
    if (rotary_dim < 2 || (rotary_dim & 1) || !freqs || !mscale) return FA_ERR_INVALID_ARG;
    if (!(base >= 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor))
        return FA_ERR_INVALID_ARG;
    if (scaling < FA_ROTARY_PLAIN || scaling > FA_ROTARY_YARN) return FA_ERR_INVALID_ARG;
    if (scaling == FA_ROTARY_YARN && (!(original_len > 0.0) || !std::isfinite(original_len)))
        return FA_ERR_INVALID_ARG;
    if (scaling == FA_ROTARY_NTK) {
        if (rotary_dim == 2) return FA_ERR_INVALID_ARG;
        base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
        if (!std::isfinite(base)) return FA_ERR_INVALID_ARG;
    }
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == FA_ROTARY_LINEAR) theta /= factor;
        if (scaling == FA_ROTARY_YARN) {
            const double turns = original_len * theta / two_pi;  // within the trained length
            double keep = (turns - 1.0) / 31.0;
            keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
            theta = theta * keep + theta / factor * (1.0 - keep);
        }
        freqs[i] = (int64_t)std::llrint(std::ldexp(theta / two_pi, 64));  // theta <= 1
    }
    *mscale = scaling == FA_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return FA_OK;
}

fa_status fa_rotary(const void* q, const void* k, void* q_out, void* k_out,
                    const fa_strides* strides, const int32_t* positions, int64_t position_stride,
                    const int64_t* freqs, int rotary_dim, float mscale, int interleaved,
                    int inverse, int B, int Hq, int Hk, int L, int D, int dtype, void* stream) {
    TraceDisarm disarm;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
    if (B < 0 || Hq < 0 || Hk < 0 || L < 0 || D <= 0) return FA_ERR_INVALID_ARG;
    if (inverse != 0 && inverse != 1) return FA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    RotaryLaunch p;
    std::memset(&p, 0, sizeof(p));
    const bool empty = B == 0 || L == 0 || (Hq == 0 && Hk == 0);
    if (rotary_dim == 0) return FA_ERR_INVALID_ARG;
    if (!empty && !freqs) return FA_ERR_INVALID_ARG;
    static const int64_t kNone[1] = {0};
    fa_status st = check_rotation(empty ? kNone : freqs, rotary_dim, mscale, interleaved, D, &p.rot);
    if (st != FA_OK) return st;
    if (empty) return FA_OK;
    if ((long long)Hq + Hk > 65535) return FA_ERR_UNSUPPORTED;
    if ((long long)B * L > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    if (!strides || position_stride < 0 || !aligned4(positions)) return FA_ERR_INVALID_ARG;
    const void* in[2] = {q, k};
    void* out[2] = {q_out, k_out};
    const int H[2] = {Hq, Hk};
    Range rin[2] = {{0, 0}, {0, 0}}, rout[2] = {{0, 0}, {0, 0}};
    for (int i = 0; i < 2; ++i) {
        RotaryOperand& o = p.op[i];
        o.H = H[i];
        if (H[i] == 0) continue;
        if (!in[i] || !out[i] || !aligned16(in[i]) || !aligned16(out[i])) return FA_ERR_INVALID_ARG;
        if (!take_strides(strides[i], B, H[i], &o.sx) ||
            !take_strides(strides[2 + i], B, H[i], &o.sy))
            return FA_ERR_INVALID_ARG;
        o.x = in[i];
        o.y = out[i];
        rin[i] = extent(in[i], o.sx, B, H[i], L, D);
        rout[i] = extent(out[i], o.sy, B, H[i], L, D);
        if (o.x != o.y) p.copy_rest = 1;
    }
    const Range rpos = positions
                           ? range(positions, ((size_t)(B - 1) * position_stride + L) * 4u)
                           : Range{0, 0};
    const Range rfreq = range(freqs, (size_t)rotary_dim / 2 * 8u);
    for (int i = 0; i < 2; ++i) {
        if (H[i] == 0) continue;
        if (overlap(rout[i], rpos) || overlap(rout[i], rfreq)) return FA_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j) {
            if (H[j] == 0) continue;
            const RotaryOperand &a = p.op[i], &b = p.op[j];
            // An output may be its own input (in place); parts of one packed tensor may interleave.
            if (overlap(rout[i], rin[j]) && !(i == j && a.y == b.x && same(a.sy, b.sx, B, a.H, L)) &&
                !packed_parts(a.y, a.sy, a.H, b.x, b.sx, b.H, B, L, D))
                return FA_ERR_INVALID_ARG;
            if (i < j && overlap(rout[i], rout[j]) && !packed_parts(a.y, a.sy, a.H, b.y, b.sy, b.H, B, L, D))
                return FA_ERR_INVALID_ARG;
        }
    }
    if (Hq == 0) {  // the kernel's first operand is never empty
        p.op[0] = p.op[1];
        p.op[1].H = 0;
    }
    p.positions = positions;
    p.pos_stride = position_stride;
    p.B = B;
    p.L = L;
    p.D = D;
    p.inverse = inverse;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return traced_launch(0, s, [&] { return launch_rotary(p, dtype == FA_BF16, s); }) == cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

fa_status fa_cache_append(const void* k, const void* v, const fa_strides* strides, void* k_cache,
                          void* v_cache, void* k_exp, void* v_exp, const int32_t* block_tables,
                          const int32_t* seq_lens, const int32_t* new_lens, const int64_t* freqs,
                          int rotary_dim, float mscale, int interleaved, int B, int H, int L, int D,
                          int num_pages, int max_pages, int dtype, int cache_dtype, void* stream) {
    TraceDisarm disarm;
    fa_status st = check_cache(B, H, L, D, num_pages, max_pages, dtype, cache_dtype);
    if (st != FA_OK) return st;
    const bool empty = B == 0 || H == 0 || L == 0;
    CacheAppendParams p;
    std::memset(&p, 0, sizeof(p));
    static const int64_t kNone[1] = {0};
    st = check_rotation(empty ? kNone : freqs, rotary_dim, mscale, interleaved, D, &p.rot);
    if (st != FA_OK) return st;
    if (empty) return FA_OK;
    if (!k || !v || !strides || !aligned16(k) || !aligned16(v) || !aligned4(new_lens))
        return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(k_cache, v_cache, k_exp, v_exp, block_tables, seq_lens, num_pages,
                           max_pages, cache_dtype))
        return FA_ERR_INVALID_ARG;
    if (!take_strides(strides[0], B, H, &p.sk) || !take_strides(strides[1], B, H, &p.sv))
        return FA_ERR_INVALID_ARG;
    const bool q8 = cache_dtype == FA_CACHE_E4M3;
    const size_t cb = cache_bytes(num_pages, H, D, cache_dtype), eb = q8 ? exp_bytes(num_pages, H) : 0;
    const Range outs[] = {range(k_cache, cb), range(v_cache, cb), range(k_exp, eb), range(v_exp, eb)};
    const Range ins[] = {extent(k, p.sk, B, H, L, D),
                         extent(v, p.sv, B, H, L, D),
                         range(block_tables, (size_t)B * max_pages * 4u),
                         range(seq_lens, (size_t)B * 4u),
                         range(new_lens, new_lens ? (size_t)B * 4u : 0),
                         range(freqs, (size_t)rotary_dim / 2 * 8u)};
    for (int a = 0; a < 4; ++a) {
        for (const Range& b : ins)
            if (overlap(outs[a], b)) return FA_ERR_INVALID_ARG;
        for (int b = a + 1; b < 4; ++b)
            if (overlap(outs[a], outs[b])) return FA_ERR_INVALID_ARG;
    }
    p.k = k;
    p.v = v;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_exp = q8 ? static_cast<uint8_t*>(k_exp) : nullptr;
    p.v_exp = q8 ? static_cast<uint8_t*>(v_exp) : nullptr;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.B = B;
    p.H = H;
    p.L = L;
    p.D = D;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.status = status_ptr();
    if (!p.status) return FA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return traced_launch(0, s, [&] { return launch_cache_append(p, dtype == FA_BF16, q8, s); }) ==
                   cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

fa_status fa_cache_read(const void* k_cache, const void* v_cache, const void* k_exp,
                        const void* v_exp, const int32_t* block_tables, const int32_t* seq_lens,
                        void* k, void* v, const fa_strides* strides, int B, int H, int L, int D,
                        int num_pages, int max_pages, int dtype, int cache_dtype, void* stream) {
    TraceDisarm disarm;
    fa_status st = check_cache(B, H, L, D, num_pages, max_pages, dtype, cache_dtype);
    if (st != FA_OK) return st;
    if (B == 0 || H == 0 || L == 0) return FA_OK;
    if (!k || !v || !strides || !aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(k_cache, v_cache, k_exp, v_exp, block_tables, seq_lens, num_pages,
                           max_pages, cache_dtype))
        return FA_ERR_INVALID_ARG;
    CacheReadParams p;
    std::memset(&p, 0, sizeof(p));
    if (!take_strides(strides[0], B, H, &p.sk) || !take_strides(strides[1], B, H, &p.sv))
        return FA_ERR_INVALID_ARG;
    const bool q8 = cache_dtype == FA_CACHE_E4M3;
    const size_t cb = cache_bytes(num_pages, H, D, cache_dtype), eb = q8 ? exp_bytes(num_pages, H) : 0;
    const Range outs[] = {extent(k, p.sk, B, H, L, D), extent(v, p.sv, B, H, L, D)};
    const Range ins[] = {range(k_cache, cb), range(v_cache, cb), range(k_exp, eb), range(v_exp, eb),
                         range(block_tables, (size_t)B * max_pages * 4u),
                         range(seq_lens, (size_t)B * 4u)};
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o, i)) return FA_ERR_INVALID_ARG;
    if (overlap(outs[0], outs[1]) && !packed_parts(k, p.sk, H, v, p.sv, H, B, L, D)) return FA_ERR_INVALID_ARG;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_exp = q8 ? static_cast<const uint8_t*>(k_exp) : nullptr;
    p.v_exp = q8 ? static_cast<const uint8_t*>(v_exp) : nullptr;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.k = k;
    p.v = v;
    p.B = B;
    p.H = H;
    p.L = L;
    p.D = D;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.status = status_ptr();
    if (!p.status) return FA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return traced_launch(0, s, [&] { return launch_cache_read(p, dtype == FA_BF16, q8, s); }) ==
                   cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

size_t fa_decode_workspace_bytes_ex(int B, int Hq, int Hk, int D, int max_pages) {
    if (B <= 0 || Hq <= 0 ||
        check_decode(B, Hq, Hk, D, 0, max_pages, 1.0f, FA_BF16, FA_CACHE_16BIT) != FA_OK)
        return 0;
    return decode_workspace(B, Hq, Hk, D, max_pages, false, 0).bytes;
}

fa_status fa_decode_paged_ex(const void* q, const void* k_cache, const void* v_cache,
                             const void* k_exp, const void* v_exp, const int32_t* block_tables,
                             const int32_t* seq_lens, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, int B, int Hq, int Hk, int D, int num_pages,
                             int max_pages, float scale, int dtype, int cache_dtype, void* stream) {
    TraceDisarm disarm;
    fa_status st = check_decode(B, Hq, Hk, D, num_pages, max_pages, scale, dtype, cache_dtype);
    if (st != FA_OK) return st;
    if (B == 0 || Hq == 0) return FA_OK;
    const bool q8 = cache_dtype == FA_CACHE_E4M3;
    if (!q || !o || !lse || !aligned16(q) || !aligned16(o) || !aligned4(lse))
        return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(k_cache, v_cache, k_exp, v_exp, block_tables, seq_lens, num_pages,
                           max_pages, cache_dtype))
        return FA_ERR_INVALID_ARG;
    GqaParams p;
    std::memset(&p, 0, sizeof(p));
    const size_t rows = (size_t)B * Hq;
    const DecodeWorkspace w = decode_workspace(B, Hq, Hk, D, max_pages, false, 0);
    const size_t ws_need = w.bytes;
    if (!workspace || workspace_bytes < ws_need || !aligned16(workspace))
        return FA_ERR_INVALID_ARG;
    const size_t cb = cache_bytes(num_pages, Hk, D, cache_dtype), eb = q8 ? exp_bytes(num_pages, Hk) : 0;
    const Range ins[] = {range(q, rows * D * 2u), range(k_cache, cb), range(v_cache, cb),
                         range(k_exp, eb), range(v_exp, eb),
                         range(block_tables, (size_t)B * max_pages * 4u),
                         range(seq_lens, (size_t)B * 4u)};
    const Range outs[] = {range(o, rows * D * 2u), range(lse, rows * 4u), range(workspace, ws_need)};
    for (int a = 0; a < 3; ++a) {
        for (const Range& in : ins)
            if (overlap(outs[a], in)) return FA_ERR_INVALID_ARG;
        for (int b = a + 1; b < 3; ++b)
            if (overlap(outs[a], outs[b])) return FA_ERR_INVALID_ARG;
    }
    if (!bind_context()) return FA_ERR_CUDA;
    if (num_pages > 0 && (!make_cache_map(&p.tm_k, k_cache, num_pages, Hk, D, dtype, q8) ||
                          !make_cache_map(&p.tm_v, v_cache, num_pages, Hk, D, dtype, q8)))
        return FA_ERR_CUDA;
    p.q = q;
    p.k_exp = static_cast<const uint8_t*>(k_exp);
    p.v_exp = static_cast<const uint8_t*>(v_exp);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.o = o;
    p.lse = lse;
    p.Hq = Hq;
    p.Hk = Hk;
    p.group = Hq / Hk;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = status_ptr();
    p.timeout_ns = wait_timeout_ns();
    if (!p.status) return FA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return run_decode(p, B, D, dtype == FA_BF16, q8, static_cast<uint8_t*>(workspace), w, 0, 0, 0,
                      s) ==
                   cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
}

size_t fa_shared_prefix_workspace_bytes(int B, int Hq, int Hk, int D, int prefix_len,
                                        int max_pages) {
    if (B <= 0 || Hq <= 0 || prefix_len < 0 || prefix_len > kMaxTokens ||
        check_decode(B, Hq, Hk, D, 0, max_pages, 1.0f, FA_BF16, FA_CACHE_16BIT) != FA_OK ||
        Hq / Hk > kTileRows)
        return 0;
    PrefixParams pp;
    prefix_plan(B, Hk, Hq / Hk, prefix_len, &pp);
    return decode_workspace(B, Hq, Hk, D, max_pages, pp.max_segments > 0, pp.max_segments).bytes;
}

fa_status fa_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* prefix_table, int prefix_len,
                                  const int32_t* block_tables, const int32_t* seq_lens, void* o,
                                  float* lse, void* workspace, size_t workspace_bytes, int B, int Hq,
                                  int Hk, int D, int num_pages, int max_pages, float scale,
                                  int dtype, void* stream) {
    TraceDisarm disarm;
    if (prefix_len < 0) return FA_ERR_INVALID_ARG;
    if (prefix_len > kMaxTokens) return FA_ERR_UNSUPPORTED;
    fa_status st = check_decode(B, Hq, Hk, D, num_pages, max_pages, scale, dtype, FA_CACHE_16BIT);
    if (st != FA_OK) return st;
    if (B == 0 || Hq == 0) return FA_OK;
    const int group = Hq / Hk;
    if (group > kTileRows) return FA_ERR_UNSUPPORTED;
    if (!q || !o || !lse || !aligned16(q) || !aligned16(o) || !aligned4(lse))
        return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(k_cache, v_cache, nullptr, nullptr, block_tables, seq_lens, num_pages,
                           max_pages, FA_CACHE_16BIT))
        return FA_ERR_INVALID_ARG;
    // A prefix needs pages to lie in.
    if (prefix_len > 0 && (!prefix_table || !aligned4(prefix_table) || num_pages == 0))
        return FA_ERR_INVALID_ARG;
    PrefixParams pp;
    std::memset(&pp, 0, sizeof(pp));
    prefix_plan(B, Hk, group, prefix_len, &pp);
    GqaParams p;
    std::memset(&p, 0, sizeof(p));
    const size_t rows = (size_t)B * Hq;
    const DecodeWorkspace w =
        decode_workspace(B, Hq, Hk, D, max_pages, pp.max_segments > 0, pp.max_segments);
    const size_t ws_need = w.bytes;
    if (!workspace || workspace_bytes < ws_need || !aligned16(workspace))
        return FA_ERR_INVALID_ARG;
    const size_t cb = cache_bytes(num_pages, Hk, D, FA_CACHE_16BIT);
    const int n_prefix_pages = prefix_len / kPageTokens + (prefix_len % kPageTokens != 0);
    const Range ins[] = {range(q, rows * D * 2u), range(k_cache, cb), range(v_cache, cb),
                         range(prefix_table, (size_t)n_prefix_pages * 4u),
                         range(block_tables, (size_t)B * max_pages * 4u),
                         range(seq_lens, (size_t)B * 4u)};
    const Range outs[] = {range(o, rows * D * 2u), range(lse, rows * 4u), range(workspace, ws_need)};
    for (int a = 0; a < 3; ++a) {
        for (const Range& in : ins)
            if (overlap(outs[a], in)) return FA_ERR_INVALID_ARG;
        for (int b = a + 1; b < 3; ++b)
            if (overlap(outs[a], outs[b])) return FA_ERR_INVALID_ARG;
    }
    if (!bind_context()) return FA_ERR_CUDA;
    if (num_pages > 0 && (!make_cache_map(&p.tm_k, k_cache, num_pages, Hk, D, dtype, false) ||
                          !make_cache_map(&p.tm_v, v_cache, num_pages, Hk, D, dtype, false)))
        return FA_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int* status = status_ptr();
    if (!status) return FA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == FA_BF16;
    int n = 0;
    if (prefix_len > 0) {
        const CUtensorMapDataType type =
            bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)B};
        const cuuint64_t qs[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * Hq * 2};
        const cuuint32_t qb[3] = {64, (cuuint32_t)group, (cuuint32_t)pp.rows_b};
        if (!make_tiled_map(&pp.tm_q, type, q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B))
            return FA_ERR_CUDA;
        pp.tm_k = p.tm_k;
        pp.tm_v = p.tm_v;
        // The last page's rows alone: what lies behind them reads as zeros.
        const int tail = prefix_len % kPageTokens;
        pp.tm_k_tail = p.tm_k;
        pp.tm_v_tail = p.tm_v;
        if (tail > 0) {
            const cuuint64_t d[3] = {(cuuint64_t)D, (cuuint64_t)tail, (cuuint64_t)num_pages * Hk};
            const cuuint64_t st2[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * kPageTokens};
            const cuuint32_t box[3] = {64, (cuuint32_t)kPageTokens, 1};
            if (!make_tiled_map(&pp.tm_k_tail, type, k_cache, 3, d, st2, box,
                                CU_TENSOR_MAP_SWIZZLE_128B) ||
                !make_tiled_map(&pp.tm_v_tail, type, v_cache, 3, d, st2, box,
                                CU_TENSOR_MAP_SWIZZLE_128B))
                return FA_ERR_CUDA;
        }
        pp.table = prefix_table;
        pp.part_o = reinterpret_cast<float*>(ws + w.prefix_o);
        pp.part_lse = reinterpret_cast<float*>(ws + w.prefix_lse);
        pp.prefix_len = prefix_len;
        pp.num_pages = num_pages;
        pp.B = B;
        pp.Hq = Hq;
        pp.Hk = Hk;
        pp.group = group;
        // The softmax takes the maximum of the stored scores: a negative scale is moved into the
        // contraction as an exact sign flip, and the multiplier keeps a masked -inf at -inf.
        pp.scale_log2 = std::fmax(std::fabs(scale) * 1.4426950408889634f, FLT_MIN);
        pp.s_negate = scale < 0.0f ? 1u : 0u;
        pp.status = status;
        pp.timeout_ns = wait_timeout_ns();
        if (traced_launch(n++, s, [&] { return launch_prefix(pp, D, bf16, s); }) != cudaSuccess)
            return FA_ERR_CUDA;
    }
    p.q = q;
    p.o = o;
    p.lse = lse;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.parts_only = prefix_len > 0;
    p.early = prefix_len > 0;
    p.Hq = Hq;
    p.Hk = Hk;
    p.group = group;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = status;
    p.timeout_ns = wait_timeout_ns();
    return run_decode(p, B, D, bf16, false, ws, w, pp.max_segments, pp.grid, n, s) == cudaSuccess ? FA_OK
                                                                                         : FA_ERR_CUDA;
}

}  // extern "C"
