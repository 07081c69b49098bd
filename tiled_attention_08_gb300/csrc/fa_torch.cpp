// fa_torch.cpp -- the operators around attention for torch tensors (host code only).
//
// The smallest of these calls run for a few microseconds on the GPU, so argument checks, output
// allocation and the autograd node are C++ here: a decode step costs the host about 9 us instead of
// 23 with the same steps in Python.  Everything else is as in the ctypes binding: the current CUDA
// stream and the caching allocator come from torch, the computation is libfa's, and a status other
// than FA_OK raises FaError(call, status).
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/_make_dual.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/fa.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

// A status of the library on its way to Python's FaError.
struct StatusError : std::exception {
    StatusError(const char* c, int s)
        : call(c), status(s), text(std::string(c) + " failed: " + fa_status_string(s)) {}
    const char* what() const noexcept override { return text.c_str(); }
    const char* call;
    int status;
    std::string text;
};
void check_status(const char* call, fa_status s) {
    if (s != FA_OK) throw StatusError(call, s);
}

int dtype_code(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return FA_BF16;
    TORCH_CHECK_TYPE(t.scalar_type() == at::kHalf, "unsupported dtype ", t.scalar_type(),
                     "; expected bfloat16 or float16");
    return FA_FP16;
}

int cuda_index(const char* name, const Tensor& t) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    return t.get_device();
}
void same_device(const char* name, const Tensor& t, int index) {
    TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == index, name, " is on ", t.device(),
                      ", expected cuda:", index);
}
void int32_vector(const char* name, const Tensor& t, int64_t n, int index) {
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n && t.is_contiguous(),
                      name, " must be a contiguous int32 [", n, "] tensor");
    same_device(name, t, index);
}

// Sizes are ints in the C interface.
int as_int(const char* name, int64_t v) {
    TORCH_CHECK_VALUE(v <= INT32_MAX, name, " is ", v, ", over 2^31 - 1");
    return (int)v;
}

// Whether the kernels can step by a view's stride of dimension i.
bool usable_stride(const Tensor& t, int i) { return t.stride(i) > 0 && (t.stride(i) & 7) == 0; }

// (batch, head, row) element strides of a [B, H, L, D] view.  The stride of a dimension of size 1 means
// nothing and may be anything: one that the library would refuse is replaced.
fa_strides row_strides(const char* name, const Tensor& t, at::IntArrayRef shape) {
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t.stride(3) == 1, name, ": the last (D) dimension must be contiguous");
    auto stride = [&](int i) { return t.size(i) > 1 || usable_stride(t, i) ? t.stride(i) : 8; };
    return {stride(0), stride(1), stride(2)};
}

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }
template <typename T = void>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* ptr(const OptTensor& t) {
    return t && t->defined() ? static_cast<T*>(t->data_ptr()) : nullptr;
}
bool given(const OptTensor& t) { return t && t->defined(); }

// Tells autograd that a caller's tensor is being written: a backward that saved it is then refused.
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(const OptTensor& t) {
    if (given(t)) written(*t);
}

// ---------------------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------------------
int rotary_dim_of(const Tensor& freqs, int index) {
    TORCH_CHECK_TYPE(freqs.scalar_type() == at::kLong && freqs.dim() == 1 && freqs.is_contiguous(),
                     "freqs must be a contiguous one-dimensional int64 tensor (rotary_freqs)");
    same_device("freqs", freqs, index);
    return as_int("rotary_dim", 2 * freqs.size(0));
}

// `t` itself where the kernels can read its rows, else a contiguous copy (an expanded gradient, for
// one, has strides of 0).
Tensor kernel_view(const Tensor& t) {
    if (t.dim() != 4) return t;
    bool ok = t.stride(3) == 1 && !(reinterpret_cast<uintptr_t>(t.data_ptr()) & 15);
    for (int i = 0; i < 3; ++i) ok = ok && (t.size(i) <= 1 || usable_stride(t, i));
    return ok ? t : t.clone(at::MemoryFormat::Contiguous);
}

struct Rotation {
    OptTensor positions;
    Tensor freqs;
    double mscale;
    bool interleaved;
};

// One or two [B, H, L, D] views turned; `outs` empty: new tensors, returned.
std::vector<Tensor> rotate(std::vector<Tensor> xs, const Rotation& r, bool inverse,
                           std::vector<Tensor> outs = {}) {
    const int index = cuda_index("x", xs[0]);
    for (const Tensor& x : xs)
        TORCH_CHECK_VALUE(x.dim() == 4, "rotary operands are [B, H, L, D] views");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    const int dt = dtype_code(xs[0]);
    const int64_t B = xs[0].size(0), L = xs[0].size(2), D = xs[0].size(3);
    const bool fresh = outs.empty();
    fa_strides st[4];
    void *in[2] = {nullptr, nullptr}, *out[2] = {nullptr, nullptr};
    int H[2] = {0, 0};
    for (size_t i = 0; i < xs.size(); ++i) {
        TORCH_CHECK_TYPE(xs[i].scalar_type() == xs[0].scalar_type(), "the operands must share a dtype");
        same_device("an operand", xs[i], index);
        const int64_t shape[4] = {B, xs[i].size(1), L, D};
        TORCH_CHECK_VALUE(xs[i].sizes() == at::IntArrayRef(shape, 4),
                          "the operands must agree in B, L and D");
        if (fresh) {
            xs[i] = kernel_view(xs[i]);
            outs.push_back(at::empty_like(xs[i]));
        } else {
            TORCH_CHECK_TYPE(outs[i].scalar_type() == xs[0].scalar_type(), "out must have the dtype of x");
            same_device("out", outs[i], index);
        }
        st[i] = row_strides("x", xs[i], at::IntArrayRef(shape, 4));
        st[2 + i] = row_strides("out", outs[i], at::IntArrayRef(shape, 4));
        in[i] = ptr(xs[i]);
        out[i] = ptr(outs[i]);
        H[i] = as_int("H", shape[1]);
    }
    if (xs.size() == 1) {
        st[1] = st[0];
        st[3] = st[2];
    }
    const int rd = rotary_dim_of(r.freqs, index);
    const int32_t* pos = nullptr;
    int64_t pos_stride = 0;
    if (given(r.positions)) {
        const Tensor& p = *r.positions;
        TORCH_CHECK_TYPE(p.scalar_type() == at::kInt, "positions must be int32");
        same_device("positions", p, index);
        const bool one = p.dim() == 1 && p.size(0) == L;
        TORCH_CHECK_VALUE((one || (p.dim() == 2 && p.size(0) == B && p.size(1) == L)) &&
                              (L <= 1 || p.stride(-1) == 1),
                          "positions must be [L] or [B, L] = (", B, ", ", L, ") with contiguous rows");
        pos = ptr<int32_t>(p);
        pos_stride = one || B <= 1 ? 0 : p.stride(0);
    }
    check_status("fa_rotary",
                 fa_rotary(in[0], in[1], out[0], out[1], st, pos, pos_stride, ptr<int64_t>(r.freqs), rd,
                           (float)r.mscale, r.interleaved, inverse, as_int("B", B), H[0], H[1],
                           as_int("L", L), as_int("D", D), dt, stream_of(index)));
    return outs;
}

// Linear in q and k (either may be missing), so the backward is the same function turned the other
// way, and can itself be differentiated.  Returns the turned ones of the two that are there.
struct Rotary : torch::autograd::Function<Rotary> {
    static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, OptTensor q,
                                                  OptTensor k, OptTensor positions, Tensor freqs,
                                                  double mscale, bool interleaved, bool inverse) {
        ctx->save_for_backward({given(positions) ? *positions : Tensor(), freqs});
        ctx->saved_data["mscale"] = mscale;
        ctx->saved_data["interleaved"] = interleaved;
        ctx->saved_data["inverse"] = inverse;
        ctx->saved_data["has_q"] = given(q);
        ctx->set_materialize_grads(false);
        std::vector<Tensor> xs;
        for (const OptTensor& x : {q, k})
            if (given(x)) xs.push_back(*x);
        return rotate(xs, {positions, freqs, mscale, interleaved}, inverse);
    }
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                   torch::autograd::variable_list grads) {
        const auto saved = ctx->get_saved_variables();
        const double mscale = ctx->saved_data["mscale"].toDouble();
        const bool interleaved = ctx->saved_data["interleaved"].toBool();
        const bool inverse = !ctx->saved_data["inverse"].toBool();
        const size_t first = ctx->saved_data["has_q"].toBool() ? 0 : 1;
        torch::autograd::variable_list out(7);
        OptTensor g[2];  // of q, of k: those that are there and wanted
        for (size_t i = 0; i < grads.size(); ++i)
            if (grads[i].defined() && ctx->needs_input_grad(i)) g[first + i] = grads[i];
        if (!g[0] && !g[1]) return out;
        const OptTensor positions = saved[0].defined() ? OptTensor(saved[0]) : OptTensor();
        torch::autograd::variable_list turned;
        if (at::GradMode::is_enabled()) {  // a graph of the gradient is wanted
            turned = Rotary::apply(g[0], g[1], positions, saved[1], mscale, interleaved, inverse);
        } else {
            std::vector<Tensor> xs;
            for (const OptTensor& x : g)
                if (x) xs.push_back(*x);
            turned = rotate(xs, {positions, saved[1], mscale, interleaved}, inverse);
        }
        size_t n = 0;
        for (int i = 0; i < 2; ++i)
            if (g[i]) out[i] = turned[n++];
        return out;
    }
};

// The operands that are there, turned; a node of the graph where one of them needs a gradient.
std::vector<Tensor> turned(const OptTensor& q, const OptTensor& k, const Rotation& r) {
    if (at::GradMode::is_enabled() && ((given(q) && q->requires_grad()) || (given(k) && k->requires_grad())))
        return Rotary::apply(q, k, r.positions, r.freqs, r.mscale, r.interleaved, false);
    std::vector<Tensor> xs;
    for (const OptTensor* x : {&q, &k})
        if (given(*x)) xs.push_back(**x);
    return rotate(xs, r, false);
}

// The tangent of a dual tensor (torch has one level of them).
OptTensor tangent_of(const Tensor& x) {
    const Tensor& t = x._fw_grad(0);
    return t.defined() && !t._is_zerotensor() ? OptTensor(t) : OptTensor();
}

std::tuple<Tensor, Tensor> rotary(const Tensor& q, const Tensor& k, const OptTensor& positions,
                                  const Tensor& freqs, double mscale, bool interleaved) {
    const Rotation r = {positions, freqs, mscale, interleaved};
    const OptTensor tq = tangent_of(q), tk = tangent_of(k);
    if (!tq && !tk) {
        const auto out = turned(q, k, r);
        return {out[0], out[1]};
    }
    // Forward mode: the map is linear, so the tangents are turned like the values.
    auto out = turned(q._fw_primal(0), k._fw_primal(0), r);
    const auto t = turned(tq, tk, r);
    size_t n = 0;
    if (tq) out[0] = at::_make_dual(out[0], t[n++], 0);
    if (tk) out[1] = at::_make_dual(out[1], t[n], 0);
    return {out[0], out[1]};
}

Tensor rotary_apply(const Tensor& x, const OptTensor& positions, const Tensor& freqs, double mscale,
                    bool interleaved, bool inverse, const OptTensor& out) {
    written(out);
    return rotate({x.detach()}, {positions, freqs, mscale, interleaved}, inverse,
                  given(out) ? std::vector<Tensor>{*out} : std::vector<Tensor>{})[0];
}

// ---------------------------------------------------------------------------------------
// The paged cache
// ---------------------------------------------------------------------------------------
struct Cache {
    int kind, num_pages, H, D;
    void *k, *v, *k_exp, *v_exp;
};

Cache check_cache(const Tensor& k, const Tensor& v, const OptTensor& ke, const OptTensor& ve,
                  at::ScalarType dtype, int index) {
    TORCH_CHECK_VALUE(k.dim() == 4 && k.size(2) == FA_PAGE_TOKENS && v.sizes() == k.sizes(),
                      "caches must be [num_pages, H, FA_PAGE_TOKENS, D]");
    TORCH_CHECK_VALUE(k.is_contiguous() && v.is_contiguous(), "the caches must be contiguous");
    same_device("k_cache", k, index);
    same_device("v_cache", v, index);
    TORCH_CHECK_TYPE(v.scalar_type() == k.scalar_type(), "k_cache and v_cache must share a dtype");
    Cache c = {FA_CACHE_16BIT, as_int("num_pages", k.size(0)), as_int("H", k.size(1)),
               as_int("D", k.size(3)), ptr(k), ptr(v), nullptr, nullptr};
    if (!given(ke) && !given(ve)) {
        TORCH_CHECK_TYPE(k.scalar_type() == dtype, "the cache holds ", k.scalar_type(),
                         ", the call's tensors ", dtype, "; an e4m3 cache needs k_exp and v_exp");
        return c;
    }
    TORCH_CHECK_TYPE(k.scalar_type() == at::kFloat8_e4m3fn,
                     "a cache with exponents must be float8_e4m3fn");
    for (const OptTensor* e : {&ke, &ve}) {
        TORCH_CHECK_VALUE(given(*e) && (*e)->scalar_type() == at::kByte &&
                              (*e)->sizes() == k.sizes().slice(0, 3) && (*e)->is_contiguous(),
                          "k_exp and v_exp must be contiguous uint8 [num_pages, H, FA_PAGE_TOKENS] tensors");
        same_device("exponents", **e, index);
    }
    c.kind = FA_CACHE_E4M3;
    c.k_exp = ptr(ke);
    c.v_exp = ptr(ve);
    return c;
}

// max_pages of a checked block table and its lengths.
int check_tables(const Tensor& block_tables, const Tensor& seq_lens, int64_t B, int index) {
    TORCH_CHECK_TYPE(block_tables.scalar_type() == at::kInt && seq_lens.scalar_type() == at::kInt,
                     "block_tables and seq_lens must be int32");
    TORCH_CHECK_VALUE(block_tables.dim() == 2 && block_tables.size(0) == B && seq_lens.dim() == 1 &&
                          seq_lens.size(0) == B,
                      "block_tables must be [B, max_pages] and seq_lens [B]");
    TORCH_CHECK_VALUE(block_tables.is_contiguous() && seq_lens.is_contiguous(),
                      "block_tables and seq_lens must be contiguous");
    same_device("block_tables", block_tables, index);
    same_device("seq_lens", seq_lens, index);
    return as_int("max_pages", block_tables.size(1));
}

void cache_append(const Tensor& k, const Tensor& v, const Tensor& k_cache, const Tensor& v_cache,
                  const Tensor& block_tables, const Tensor& seq_lens, const OptTensor& new_lens,
                  const OptTensor& k_exp, const OptTensor& v_exp, const OptTensor& freqs, double mscale,
                  bool interleaved) {
    const int index = cuda_index("k", k);
    const int dt = dtype_code(k);
    TORCH_CHECK_VALUE(k.dim() == 4, "k and v must be [B, H, L, D] views");
    const fa_strides st[2] = {row_strides("k", k, k.sizes()), row_strides("v", v, k.sizes())};
    TORCH_CHECK_TYPE(v.scalar_type() == k.scalar_type(), "k and v must share a dtype");
    same_device("v", v, index);
    const int64_t B = k.size(0);
    const Cache c = check_cache(k_cache, v_cache, k_exp, v_exp, k.scalar_type(), index);
    TORCH_CHECK_VALUE(c.H == k.size(1) && c.D == k.size(3), "the cache has ", c.H, " heads of ", c.D,
                      ", k has ", k.size(1), " of ", k.size(3));
    const int max_pages = check_tables(block_tables, seq_lens, B, index);
    if (given(new_lens)) int32_vector("new_lens", *new_lens, B, index);
    const int rd = given(freqs) ? rotary_dim_of(*freqs, index) : 0;
    written(k_cache);
    written(v_cache);
    written(k_exp);
    written(v_exp);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    check_status("fa_cache_append",
                 fa_cache_append(ptr(k), ptr(v), st, c.k, c.v, c.k_exp, c.v_exp,
                                 ptr<int32_t>(block_tables), ptr<int32_t>(seq_lens),
                                 ptr<int32_t>(new_lens), ptr<int64_t>(freqs), rd, (float)mscale,
                                 interleaved, as_int("B", B), c.H, as_int("L", k.size(2)), c.D,
                                 c.num_pages, max_pages, dt, c.kind, stream_of(index)));
}

std::tuple<Tensor, Tensor> cache_read(const Tensor& k_cache, const Tensor& v_cache,
                                      const Tensor& block_tables, const Tensor& seq_lens,
                                      int64_t length, const OptTensor& k_exp, const OptTensor& v_exp,
                                      std::optional<at::ScalarType> dtype, const OptTensor& out_k,
                                      const OptTensor& out_v) {
    const int index = cuda_index("k_cache", k_cache);
    const at::ScalarType type = dtype ? *dtype : given(out_k) ? out_k->scalar_type() : k_cache.scalar_type();
    TORCH_CHECK_VALUE(seq_lens.dim() == 1 && length >= 0, "seq_lens must be [B], length at least 0");
    const Cache c = check_cache(k_cache, v_cache, k_exp, v_exp, type, index);
    const int64_t B = seq_lens.size(0);
    const int max_pages = check_tables(block_tables, seq_lens, B, index);
    const int64_t shape[4] = {B, c.H, length, c.D};
    const at::IntArrayRef sizes(shape, 4);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    const auto opt = k_cache.options().dtype(type);
    const Tensor k = given(out_k) ? *out_k : at::empty(sizes, opt);
    const Tensor v = given(out_v) ? *out_v : at::empty(sizes, opt);
    TORCH_CHECK_TYPE(k.scalar_type() == type && v.scalar_type() == type, "out must have the call's dtype");
    const int dt = dtype_code(k);
    same_device("out[0]", k, index);
    same_device("out[1]", v, index);
    TORCH_CHECK_VALUE(k.dim() == 4 && v.dim() == 4, "out must be [B, H, length, D] views");
    const fa_strides st[2] = {row_strides("out[0]", k, sizes), row_strides("out[1]", v, sizes)};
    written(out_k);
    written(out_v);
    check_status("fa_cache_read",
                 fa_cache_read(c.k, c.v, c.k_exp, c.v_exp, ptr<int32_t>(block_tables),
                               ptr<int32_t>(seq_lens), ptr(k), ptr(v), st, as_int("B", B), c.H,
                               as_int("length", length), c.D, c.num_pages, max_pages, dt, c.kind,
                               stream_of(index)));
    return {k, v};
}

// ---------------------------------------------------------------------------------------
// Decode steps
// ---------------------------------------------------------------------------------------
struct Step {
    int index, dt, B, Hq, D;
    Tensor o, lse;
};
Step decode_outputs(const Tensor& q, const OptTensor& out, const OptTensor& lse) {
    const int index = cuda_index("q", q);
    TORCH_CHECK_VALUE(q.dim() == 3 && q.is_contiguous(), "q must be a contiguous [B, H, D] tensor");
    Step s = {index, dtype_code(q), as_int("B", q.size(0)), as_int("H", q.size(1)),
              as_int("D", q.size(2)), {}, {}};
    if (given(out)) {
        TORCH_CHECK_VALUE(out->scalar_type() == q.scalar_type() && out->sizes() == q.sizes() &&
                              out->is_contiguous(),
                          "out must be a contiguous tensor like q");
        same_device("out", *out, index);
        written(*out);
        s.o = *out;
    } else {
        s.o = at::empty(q.sizes(), q.options());
    }
    if (given(lse)) {
        TORCH_CHECK_VALUE(lse->scalar_type() == at::kFloat && lse->sizes() == q.sizes().slice(0, 2) &&
                              lse->is_contiguous(),
                          "lse must be a contiguous fp32 [B, H] tensor");
        same_device("lse", *lse, index);
        written(*lse);
        s.lse = *lse;
    } else {
        s.lse = at::empty(q.sizes().slice(0, 2), q.options().dtype(at::kFloat));
    }
    return s;
}

// The caller's workspace, or a new one where any is needed.
Tensor workspace_of(const OptTensor& workspace, size_t need, const Tensor& q, int index) {
    if (given(workspace)) {
        same_device("workspace", *workspace, index);
        TORCH_CHECK_VALUE(workspace->is_contiguous(), "workspace must be contiguous");
        written(*workspace);
        return *workspace;
    }
    return at::empty({(int64_t)need}, q.options().dtype(at::kByte));
}

float scale_of(const std::optional<double>& scale, int D) {
    return (float)(scale ? *scale : 1.0 / std::sqrt((double)D));
}

std::tuple<Tensor, Tensor> decode_paged_ex(const Tensor& q, const Tensor& k_cache, const Tensor& v_cache,
                                           const Tensor& block_tables, const Tensor& seq_lens,
                                           std::optional<double> scale, const OptTensor& out,
                                           const OptTensor& lse, const OptTensor& workspace,
                                           const OptTensor& k_exp, const OptTensor& v_exp) {
    const c10::cuda::OptionalCUDAGuard guard(at::device_of(q));
    const Step s = decode_outputs(q, out, lse);
    const Cache c = check_cache(k_cache, v_cache, k_exp, v_exp, q.scalar_type(), s.index);
    TORCH_CHECK_VALUE(c.D == s.D, "the cache has heads of ", c.D, ", q of ", s.D);
    const int max_pages = check_tables(block_tables, seq_lens, s.B, s.index);
    const Tensor ws = workspace_of(
        workspace, fa_decode_workspace_bytes_ex(s.B, s.Hq, c.H, s.D, max_pages), q, s.index);
    check_status("fa_decode_paged_ex",
                 fa_decode_paged_ex(ptr(q), c.k, c.v, c.k_exp, c.v_exp, ptr<int32_t>(block_tables),
                                    ptr<int32_t>(seq_lens), ptr(s.o), ptr<float>(s.lse), ptr(ws),
                                    ws.nbytes(), s.B, s.Hq, c.H, s.D, c.num_pages, max_pages,
                                    scale_of(scale, s.D), s.dt, c.kind, stream_of(s.index)));
    return {s.o, s.lse};
}

// A caller's buffer that holds at least n elements of a type.
void check_room(const char* name, const Tensor& t, at::ScalarType type, int64_t n, int index) {
    same_device(name, t, index);
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.is_contiguous() && t.numel() >= n, name,
                      " must be a contiguous ", type, " tensor of at least ", n, " elements");
}

// decode_paged: the kernel of equal heads over a 16-bit cache where the call has that form, else
// fa_decode_paged_ex.  That form also takes buffers made for more sequences than q has: tables, lengths
// and outputs with more rows, of which the first B are used, in any shape.
std::tuple<Tensor, Tensor> decode_paged(const Tensor& q, const Tensor& k_cache, const Tensor& v_cache,
                                        const Tensor& block_tables, const Tensor& seq_lens,
                                        std::optional<double> scale, const OptTensor& out,
                                        const OptTensor& lse, const OptTensor& workspace,
                                        const OptTensor& k_exp, const OptTensor& v_exp) {
    if (given(k_exp) || given(v_exp) || q.dim() != 3 || k_cache.dim() != 4 || k_cache.size(1) != q.size(1))
        return decode_paged_ex(q, k_cache, v_cache, block_tables, seq_lens, scale, out, lse, workspace,
                               k_exp, v_exp);
    const c10::cuda::OptionalCUDAGuard guard(at::device_of(q));
    const int index = cuda_index("q", q);
    TORCH_CHECK_VALUE(q.is_contiguous(), "q must be contiguous");
    const int dt = dtype_code(q);
    const Cache c = check_cache(k_cache, v_cache, {}, {}, q.scalar_type(), index);
    const int B = as_int("B", q.size(0)), D = as_int("D", q.size(2));
    TORCH_CHECK_VALUE(c.D == D, "the cache has heads of ", c.D, ", q of ", D);
    TORCH_CHECK_TYPE(block_tables.scalar_type() == at::kInt && seq_lens.scalar_type() == at::kInt,
                     "block_tables and seq_lens must be int32");
    TORCH_CHECK_VALUE(block_tables.dim() == 2, "block_tables must be [B, max_pages]");
    const int max_pages = as_int("max_pages", block_tables.size(1));
    check_room("block_tables", block_tables, at::kInt, (int64_t)B * max_pages, index);
    check_room("seq_lens", seq_lens, at::kInt, B, index);
    if (given(out)) check_room("out", *out, q.scalar_type(), q.numel(), index);
    if (given(lse)) check_room("lse", *lse, at::kFloat, (int64_t)B * c.H, index);
    const Tensor o = given(out) ? *out : at::empty(q.sizes(), q.options());
    const Tensor l = given(lse) ? *lse : at::empty({B, c.H}, q.options().dtype(at::kFloat));
    written(out);
    written(lse);
    const Tensor ws =
        workspace_of(workspace, fa_decode_workspace_bytes(B, c.H, D, max_pages), q, index);
    check_status("fa_decode_paged",
                 fa_decode_paged(ptr(q), c.k, c.v, ptr<int32_t>(block_tables), ptr<int32_t>(seq_lens),
                                 ptr(o), ptr<float>(l), ptr(ws), ws.nbytes(), B, c.H, D, c.num_pages,
                                 max_pages, scale_of(scale, D), dt, stream_of(index)));
    return {o, l};
}

std::tuple<Tensor, Tensor> decode_shared_prefix(const Tensor& q, const Tensor& k_cache,
                                                const Tensor& v_cache, const Tensor& prefix_table,
                                                int64_t prefix_len, const Tensor& block_tables,
                                                const Tensor& seq_lens, std::optional<double> scale,
                                                const OptTensor& out, const OptTensor& lse,
                                                const OptTensor& workspace) {
    const c10::cuda::OptionalCUDAGuard guard(at::device_of(q));
    const Step s = decode_outputs(q, out, lse);
    const Cache c = check_cache(k_cache, v_cache, {}, {}, q.scalar_type(), s.index);
    TORCH_CHECK_VALUE(c.D == s.D, "the cache has heads of ", c.D, ", q of ", s.D);
    const int max_pages = check_tables(block_tables, seq_lens, s.B, s.index);
    TORCH_CHECK_TYPE(prefix_table.scalar_type() == at::kInt && prefix_table.dim() == 1 &&
                         prefix_table.is_contiguous(),
                     "prefix_table must be a contiguous one-dimensional int32 tensor");
    same_device("prefix_table", prefix_table, s.index);
    TORCH_CHECK_VALUE(prefix_len >= 0 && prefix_len <= FA_PAGE_TOKENS * prefix_table.size(0),
                      "prefix_table has room for ", FA_PAGE_TOKENS * prefix_table.size(0),
                      " tokens, not ", prefix_len);
    const int n = as_int("prefix_len", prefix_len);
    const Tensor ws = workspace_of(
        workspace, fa_shared_prefix_workspace_bytes(s.B, s.Hq, c.H, s.D, n, max_pages), q, s.index);
    check_status("fa_decode_shared_prefix",
                 fa_decode_shared_prefix(ptr(q), c.k, c.v, ptr<int32_t>(prefix_table), n,
                                         ptr<int32_t>(block_tables), ptr<int32_t>(seq_lens), ptr(s.o),
                                         ptr<float>(s.lse), ptr(ws), ws.nbytes(), s.B, s.Hq, c.H, s.D,
                                         c.num_pages, max_pages, scale_of(scale, s.D), s.dt,
                                         stream_of(s.index)));
    return {s.o, s.lse};
}

PyObject* status_error_class = nullptr;

}  // namespace

PYBIND11_MODULE(fa_torch, m) {
    m.def("set_error", [](const py::object& cls) {  // FaError(call, status), once
        status_error_class = cls.inc_ref().ptr();
        py::register_exception_translator([](std::exception_ptr p) {
            try {
                if (p) std::rethrow_exception(p);
            } catch (const StatusError& e) {
                const py::object v = py::reinterpret_borrow<py::object>(status_error_class)(e.call, e.status);
                PyErr_SetObject(status_error_class, v.ptr());
            }
        });
    });
    m.def("rotary", &rotary);
    m.def("rotary_apply", &rotary_apply);
    m.def("cache_append", &cache_append);
    m.def("cache_read", &cache_read);
    m.def("decode_paged", &decode_paged);
    m.def("decode_paged_ex", &decode_paged_ex);
    m.def("decode_shared_prefix", &decode_shared_prefix);
}
