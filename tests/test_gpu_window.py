"""Attention under a sliding window with first tokens that stay visible: forward and gradients against
the definition in 64 bits, with tolerances derived in window_reference."""
import math

import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from window_reference import reference, sees, within

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def status():
    return fa.fa_get_device_status(torch.cuda.current_stream().cuda_stream)


def operands(seed, B, Hq, Hk, Lq, Lk, D, dtype, layout="bhld"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def new(H, L):
        if layout == "blhd":
            return torch.randn(B, L, H, D, generator=g, device="cuda", dtype=dtype).transpose(1, 2)
        return torch.randn(B, H, L, D, generator=g, device="cuda", dtype=dtype)

    if layout == "packed":  # [B, L, Hq + 2 Hk, D]
        x = torch.randn(B, Lq, Hq + 2 * Hk, D, generator=g, device="cuda", dtype=dtype).transpose(1, 2)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    else:
        q, k, v = new(Hq, Lq), new(Hk, Lk), new(Hk, Lk)
    return q, k, v, new(Hq, Lq)


def check(out, q, k, v, do, window, sinks, scale):
    """out: dict of o, lse (and dq, dk, dv)."""
    B, Hq, Lq, D = q.shape
    Hk, Lk = k.shape[1:3]
    G = Hq // Hk
    mask = sees(Lq, Lk, window, sinks)
    for b in range(B):
        for h in range(Hk):
            heads = slice(h * G, h * G + G)
            want = reference(q[b, heads], k[b, h], v[b, h], mask, scale, do[b, heads] if "dq" in out else None)
            for name, vb in want.items():
                if name in out:
                    got = out[name][b, h] if name in ("dk", "dv") else out[name][b, heads]
                    within(got, vb, f"{name}[{b}, {h}]")


def run(q, k, v, do, window, sinks, scale=None):
    o, lse = fa.window_forward(q, k, v, window, sinks, scale)
    dq, dk, dv = fa.window_backward(q, k, v, o, lse, do, window, sinks, scale)
    assert status() == fa.FA_OK
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


# B, Hq, Hk, Lq, Lk, D, dtype, layout, window, sinks
CASES = [
    (1, 1, 1, 1, 1, 64, BF16, "bhld", 1, 0),
    (2, 2, 1, 1, 300, 128, FP16, "bhld", 128, 4),          # one token behind 299
    (1, 2, 2, 127, 127, 64, FP16, "blhd", 16, 3),
    (1, 4, 2, 128, 128, 128, BF16, "bhld", 128, 0),
    (1, 3, 1, 129, 129, 128, BF16, "bhld", 64, 1),         # an odd group
    (2, 6, 2, 300, 300, 64, BF16, "packed", 100, 7),
    (1, 8, 1, 513, 513, 128, FP16, "blhd", 129, 130),      # first tokens past a tile
    (1, 2, 2, 1000, 1000, 64, FP16, "bhld", 1, 0),         # each sees itself alone
    (1, 2, 1, 1000, 1000, 128, BF16, "packed", 2, 1),
    (1, 1, 1, 700, 700, 128, FP16, "bhld", 5000, 0),       # the causal mask
    (1, 2, 2, 700, 700, 64, BF16, "bhld", 300, 5000),      # every key a first token
    (2, 4, 4, 257, 900, 128, BF16, "blhd", 256, 0),        # behind earlier keys that nobody sees
    (1, 4, 1, 257, 900, 64, FP16, "bhld", 256, 200),
    (1, 4, 2, 900, 257, 128, FP16, "bhld", 128, 5),        # 643 rows that see nothing
    (1, 3, 3, 900, 257, 64, BF16, "blhd", 7, 0),
    (1, 5, 5, 640, 640, 128, BF16, "bhld", 127, 128),
    (3, 16, 4, 1100, 1100, 64, FP16, "blhd", 250, 131),
    # More query tiles than SMs: two heads, or two tiles, at a time.
    (2, 9, 3, 1500, 1500, 64, BF16, "bhld", 200, 10),
    (1, 24, 24, 1024, 1024, 128, FP16, "blhd", 256, 1),
    (2, 16, 8, 700, 1900, 128, BF16, "bhld", 333, 0),
    (3, 10, 2, 1900, 700, 64, FP16, "bhld", 333, 140),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[1]}of{c[2]}_L{c[3]}x{c[4]}_D{c[5]}_w{c[8]}_s{c[9]}" for c in CASES])
def test_forward_and_gradients(case):
    B, Hq, Hk, Lq, Lk, D, dtype, layout, window, sinks = case
    q, k, v, do = operands(1, B, Hq, Hk, Lq, Lk, D, dtype, layout)
    check(run(q, k, v, do, window, sinks), q, k, v, do, window, sinks, 1 / math.sqrt(D))


def test_first_tokens_cut_into_parts():
    """One head, a long sequence and a short window: the first tokens' tiles are seen by 64 query tiles, every
    other by two, and are cut into parts (the workspace says so)."""
    B, Hq, Hk, L, D, window, sinks = 1, 2, 1, 8190, 64, 60, 150
    assert fa.fa_window_bwd_workspace_bytes(B, Hq, Hk, L, L, D, window, sinks) > \
        fa.fa_window_bwd_workspace_bytes(B, Hq, Hk, L, L, D, window, 0)
    q, k, v, do = operands(2, B, Hq, Hk, L, L, D, BF16)
    out = run(q, k, v, do, window, sinks)
    check(out, q, k, v, do, window, sinks, 1 / math.sqrt(D))
    again = run(q, k, v, do, window, sinks)
    assert all(torch.equal(out[x], again[x]) for x in out)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_scales(scale):
    q, k, v, do = operands(3, 1, 4, 2, 300, 300, 64, FP16)
    check(run(q, k, v, do, 90, 9, scale), q, k, v, do, 90, 9, scale)


def test_far_apart_scores():
    """Rows whose hidden keys would dominate: no hidden score may leak into a maximum or a sum, and an
    exponential of one must not overflow."""
    q, k, v, do = operands(4, 1, 2, 1, 600, 600, 128, BF16)
    k[:, :, ::3] *= 40
    q[:, :, 100:300] *= 8
    check(run(q, k, v, do, 70, 3), q, k, v, do, 70, 3, 1 / math.sqrt(128))


def test_a_window_of_all_keys_is_the_causal_mask():
    q, k, v, _ = operands(5, 2, 4, 4, 500, 500, 128, BF16)
    o, lse = fa.window_forward(q, k, v, 500)
    want, want_lse = fa.forward(q, k, v, causal=True)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_rows_that_see_nothing_and_keys_that_nobody_sees():
    q, k, v, do = operands(6, 1, 2, 1, 300, 100, 64, FP16)
    out = run(q, k, v, do, 30, 0)
    assert not out["o"][:, :, :200].any() and not out["dq"][:, :, :200].any()
    assert (out["lse"][:, :, :200] == -math.inf).all()
    q, k, v, do = operands(7, 1, 2, 1, 100, 700, 64, FP16)
    out = run(q, k, v, do, 30, 3)
    seen = sees(100, 700, 30, 3).any(0)
    for x in ("dk", "dv"):
        assert not out[x][:, :, ~seen].any() and out[x][:, :, seen].any()


def test_autograd_matches_the_calls():
    q, k, v, do = operands(8, 2, 6, 2, 333, 333, 128, BF16, "packed")
    want = run(q, k, v, do, 77, 5)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = fa.attention_window(*leaves, 77, 5)
    got = torch.autograd.grad(o, leaves, do)
    assert torch.equal(o, want["o"])
    assert all(torch.equal(a, want[n]) for a, n in zip(got, ("dq", "dk", "dv")))
    with torch.no_grad():
        assert torch.equal(fa.attention_window(*leaves, 77, 5), want["o"])


def test_broadcast_inputs_and_gradients():
    """One key head for the whole batch, expanded, and a gradient of ones (strides of 0)."""
    q, k, v, _ = operands(9, 3, 2, 2, 150, 150, 64, FP16)
    k, v = (x[:1].clone().requires_grad_() for x in (k, v))
    q.requires_grad_()
    fa.attention_window(q, k.expand(3, 2, 150, 64), v.expand(3, 2, 150, 64), 40, 2).sum().backward()
    full = [x.detach().repeat(3, 1, 1, 1) for x in (k, v)]
    o, lse = fa.window_forward(q.detach(), *full, 40, 2)
    dq, dk, dv = fa.window_backward(q.detach(), *full, o, lse, torch.ones_like(o), 40, 2)
    assert torch.equal(q.grad, dq)
    for got, parts in ((k.grad, dk), (v.grad, dv)):
        want = parts.double().sum(0, keepdim=True)
        bound = torch.finfo(FP16).eps * parts.double().abs().sum(0, keepdim=True) + 2.0 ** -24
        assert ((got.double() - want).abs() <= bound).all()


def test_gradients_against_differences():
    """sum(o * do) along a direction, from the operator's own forward in both directions: its gradient is
    the slope.  The step is 2^-4 of the inputs; the slope's error is the curvature term (third
    derivative, bounded by comparison with half the step) and the rounding of O over the step."""
    q, k, v, do = operands(10, 1, 4, 2, 200, 200, 64, FP16)
    out = run(q, k, v, do, 50, 4)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    for which, x in enumerate((q, k, v)):
        step = (torch.randn(x.shape, generator=g, device="cuda") / 16).to(FP16).float()

        def f(h):
            a = [y.float() for y in (q, k, v)]
            a[which] = a[which] + h * step
            mask = sees(200, 200, 50, 4)
            qq, kk, vv = (y.double() for y in a)
            kk, vv = (y.repeat_interleave(2, 1) for y in (kk, vv))
            p = torch.softmax(torch.where(mask, qq @ kk.mT / 8, -math.inf), -1)
            return float((p @ vv * do.double()).sum())

        full, half = (f(1) - f(-1)) / 2, f(0.5) - f(-0.5)
        slope = half + (half - full) / 3  # the third derivative taken out
        grad = out[("dq", "dk", "dv")[which]].double()
        got = float((grad * step.double()).sum())
        # A gradient's elements are each within about 2 eps of their terms' magnitude, independent of
        # the direction: the sum's error is at most that of all of them with one sign.
        bound = 2 * torch.finfo(FP16).eps * float((grad.abs() * step.abs().double()).sum()) * 4 + \
            abs(half - full) / 8 + 1e-6
        assert abs(got - slope) <= bound, (which, got, slope, bound)


def test_captured_in_a_graph_and_replayed():
    q, k, v, do = operands(12, 1, 4, 2, 700, 700, 64, BF16)
    s = torch.cuda.Stream()
    ws = torch.empty(fa.fa_window_bwd_workspace_bytes(1, 4, 2, 700, 700, 64, 100, 9), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 4, 700, device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]

    def step():
        fa.window_forward(q, k, v, 100, 9, out=o, lse=lse)
        fa.window_backward(q, k, v, o, lse, do, 100, 9, workspace=ws, grads=grads)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    new = operands(13, 1, 4, 2, 700, 700, 64, BF16)
    for x, y in zip((q, k, v, do), new):
        x.copy_(y)
    for x in (o, lse, *grads):
        x.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    want = run(q, k, v, do, 100, 9)
    for got, n in zip((o, lse, *grads), ("o", "lse", "dq", "dk", "dv")):
        assert torch.equal(got, want[n]), n


def test_strides_past_31_bits():
    """A batch stride of more than 2^31 elements (rows far apart in one buffer)."""
    far = (1 << 31) + 1024
    buf = torch.empty(far + 4 * 300 * 64, device="cuda", dtype=BF16)

    def at(first):
        return buf.as_strided((2, 1, 300, 64), (far, 300 * 64, 64, 1), first)

    q, k, v, do = operands(14, 2, 1, 1, 300, 300, 64, BF16)
    want = run(q, k, v, do, 64, 2)
    fq, fk, fv = at(0), at(300 * 64), at(2 * 300 * 64)
    for x, y in ((fq, q), (fk, k), (fv, v)):
        x.copy_(y)
    fo = at(3 * 300 * 64)
    o, lse = fa.window_forward(fq, fk, fv, 64, 2, out=fo)
    got = fa.window_backward(fq, fk, fv, o, lse, do, 64, 2)
    assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])
    assert all(torch.equal(a, want[n]) for a, n in zip(got, ("dq", "dk", "dv")))


def test_on_a_side_stream():
    q, k, v, do = operands(15, 1, 2, 1, 400, 400, 128, BF16)
    want = run(q, k, v, do, 90, 3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        leaves = [x.detach().requires_grad_() for x in (q, k, v)]
        o = fa.attention_window(*leaves, 90, 3)
        got = torch.autograd.grad(o, leaves, do)
    s.synchronize()
    assert torch.equal(o, want["o"])
    assert all(torch.equal(a, want[n]) for a, n in zip(got, ("dq", "dk", "dv")))


def test_refusals():
    q, k, v, do = operands(16, 1, 4, 2, 64, 64, 64, BF16)
    for window, sinks in ((0, 0), (-1, 0), (5, -1)):
        with pytest.raises(fa.FaError):
            fa.window_forward(q, k, v, window, sinks)
    with pytest.raises(fa.FaError):  # heads that do not divide
        fa.window_forward(q[:, :3], k, v, 4)
    with pytest.raises(ValueError):
        fa.window_forward(q, k[..., :32], v, 4)
    with pytest.raises(ValueError):
        fa.window_forward(q, k, v[:, :1], 4)
    with pytest.raises(TypeError):
        fa.window_forward(q, k.half(), v, 4)
    with pytest.raises(TypeError):
        fa.window_forward(q.float(), k.float(), v.float(), 4)
    with pytest.raises(ValueError):
        fa.window_forward(q, k.cpu(), v, 4)
    o, lse = fa.window_forward(q, k, v, 4)
    with pytest.raises(fa.FaError):  # out is an input
        fa.window_forward(q, k, v, 4, out=q)
    with pytest.raises(fa.FaError):
        fa.window_backward(q, k, v, o, lse, do, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.window_backward(q, k, v, o, lse[:, :2], do, 4)
    q.requires_grad_()
    o = fa.attention_window(q, k, v, 4)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(o, q, do, create_graph=True)
    assert status() == fa.FA_OK


def test_empty_and_query_free_calls():
    q, k, v, _ = operands(17, 1, 2, 1, 0, 50, 64, BF16)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = fa.attention_window(*leaves, 4)
    assert o.shape == q.shape
    o.sum().backward()
    assert not leaves[1].grad.any() and not leaves[2].grad.any()
    with pytest.raises(fa.FaError):
        fa.window_forward(*operands(18, 1, 2, 1, 5, 0, 64, BF16)[:3], 4)
    q, k, v, _ = operands(17, 1, 0, 1, 9, 9, 64, BF16)  # no query head
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    fa.attention_window(*leaves, 4).sum().backward()
    assert not leaves[1].grad.any() and not leaves[2].grad.any()


def test_a_saved_input_that_is_written_is_noticed():
    q, k, v, do = operands(19, 1, 2, 1, 64, 64, 64, BF16)
    q.requires_grad_()
    o = fa.attention_window(q, k, v, 8)
    k.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(o, q, do)
