"""Rotary positions (fa_rotary) against the definition in 64 bits, through the public calls.

Tolerance.  The exact reduction leaves under 2^-33 turns for positions below 2^31; the angle, at
most an eighth of a turn once the nearest quarter is split off, and its sine and cosine are each
within a few units of 2^-24, and so are the products and the sum.  A result y = x1 c - x2 s is
therefore off by well under 1.5e-6 (|x1| + |x2|) mscale (25 units of 2^-24) before its one
rounding to 16 bits, which is off by half a step: eps/2 of the value (and half the smallest
subnormal, 2^-25, in fp16).
"""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def thetas(rd, base=10000.0, scaling="none", factor=1.0, original=0.0):
    i = np.arange(rd // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rd / (rd - 2))
    th = base ** (-2.0 * i / rd)
    if scaling == "linear":
        th = th / factor
    if scaling == "yarn":
        keep = np.clip((original * th / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
        th = th * keep + th / factor * (1.0 - keep)
    return th, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def reference(x, pos, th, mscale, inter, inverse=False):
    """(y, |x1| + |x2| of each element's pair, 0 past the rotated part); x [B,H,L,D], pos [B,L]."""
    x = gh.f64(x)
    r = 2 * len(th)
    ang = pos.astype(np.float64)[:, None, :, None] * th * (-1.0 if inverse else 1.0)
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
    y, mag = x.copy(), np.zeros_like(x)
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def check(got, x, pos, th, mscale, inter, inverse=False):
    y, mag = reference(x, pos, th, mscale, inter, inverse)
    half = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    bound = half * np.abs(y) + 1.5e-6 * mscale * mag * (1 + half) + tiny
    err = np.abs(gh.f64(got) - y)
    assert np.all(err <= bound), float((err - bound).max())
    r = 2 * len(th)
    assert torch.equal(got[..., r:], x[..., r:])  # elements past the rotated part: copied


def randn(*shape, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


@pytest.mark.parametrize("B,Hq,Hk,L,D,rd,inter,dtype", [
    (2, 4, 2, 33, 128, 128, False, torch.bfloat16),
    (1, 3, 1, 1, 64, 64, False, torch.float16),
    (3, 5, 5, 7, 64, 32, True, torch.bfloat16),
    (2, 2, 1, 130, 128, 96, False, torch.float16),   # 16-byte units, part of the head
    (1, 17, 3, 9, 128, 104, True, torch.float16),
    (2, 2, 2, 5, 128, 40, False, torch.bfloat16),    # pairs that cross 16-byte units
    (2, 1, 1, 6, 64, 2, False, torch.bfloat16),
    (1, 2, 2, 11, 64, 20, True, torch.float16),
    (1, 1, 1, 1, 128, 2, True, torch.bfloat16),
], ids=str)
def test_rotary_shapes(B, Hq, Hk, L, D, rd, inter, dtype):
    q, k = randn(B, Hq, L, D, dtype=dtype), randn(B, Hk, L, D, dtype=dtype, seed=1)
    th, _ = thetas(rd)
    freqs, mscale = fa.rotary_freqs(rd)
    rng = np.random.default_rng(B * 100 + L)
    pos = rng.integers(0, 5000, (B, L)).astype(np.int32)
    qo, ko = fa.rotary(q, k, torch.from_numpy(pos).cuda(), freqs, mscale, inter)
    check(qo, q, pos, th, mscale, inter)
    check(ko, k, pos, th, mscale, inter)
    row = torch.from_numpy(pos[0]).cuda()  # one row of positions for every sequence
    qo, _ = fa.rotary(q, k, row, freqs, mscale, inter)
    check(qo, q, np.repeat(pos[:1], B, 0), th, mscale, inter)
    ko = fa.rotary_apply(k, None, freqs, mscale, inter, inverse=True)  # positions 0 .. L-1
    check(ko, k, np.repeat(np.arange(L)[None], B, 0), th, mscale, inter, inverse=True)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 4.0),
                                            ("yarn", 16.0)])
def test_rotary_far_positions_and_scalings(scaling, factor):
    """Positions up to 2^31 - 1 and negative ones: angles reduced without loss."""
    rd, D = 64, 64
    th, m = thetas(rd, 500000.0, scaling, factor, 4096)
    freqs, mscale = fa.rotary_freqs(rd, 500000.0, scaling, factor, original_len=4096)
    assert abs(mscale - m) <= 1e-6
    pos = np.array([[0, 1, 4095, 131071, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -1, -77777,
                     -(1 << 31)]], dtype=np.int64)
    x = randn(1, 3, pos.shape[1], D, dtype=torch.float16, seed=3)
    got = fa.rotary_apply(x, torch.from_numpy(pos.astype(np.int32)).cuda(), freqs, mscale)
    # 64-bit reference angles at 2^31: reduce by turns in extended precision.
    turns = pos.astype(np.longdouble)[..., None] * (th.astype(np.longdouble) / (2 * np.longdouble(math.pi)))
    ang = ((turns - np.round(turns)) * 2 * np.longdouble(math.pi)).astype(np.float64)
    xr = gh.f64(x)
    a, b = xr[..., :32], xr[..., 32:]
    c, s = np.cos(ang)[:, None] * m, np.sin(ang)[:, None] * m
    ref = np.concatenate((a * c - b * s, b * c + a * s), -1)
    mag = np.concatenate((np.abs(a) + np.abs(b),) * 2, -1)
    # theta / (2 pi) is held to a relative 2^-52 (its fp64 quotient) and 2^-65 turns.
    far = np.abs(pos.astype(np.float64))[:, None, :, None] * (np.concatenate((th, th)) * 2.0 ** -51 + 2.0 ** -62)
    bound = 2.0 ** -11 * np.abs(ref) + (1.5e-6 + 2 * far) * m * mag + 2.0 ** -25
    assert np.all(np.abs(gh.f64(got) - ref) <= bound)


def test_rotary_layouts_and_in_place():
    """[B, L, H, D] views, the parts of a packed tensor, and in place through them."""
    B, L, H, D = 2, 37, 3, 64
    freqs, mscale = fa.rotary_freqs(D)
    th, _ = thetas(D)
    pos = np.repeat(np.arange(L)[None], B, 0)
    x = randn(B, L, 3, H, D, dtype=torch.bfloat16)
    q, k = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
    qo, ko = fa.rotary(q, k, None, freqs, mscale)
    check(qo, q, pos, th, mscale, False)
    check(ko, k, pos, th, mscale, False)
    y = x.clone()
    yq, yk = y[:, :, 0].transpose(1, 2), y[:, :, 1].transpose(1, 2)
    fa.rotary_apply(yq, None, freqs, mscale, out=yq)
    fa.rotary_apply(yk, None, freqs, mscale, out=yk)
    assert torch.equal(yq, qo) and torch.equal(yk, ko) and torch.equal(y[:, :, 2], x[:, :, 2])
    with pytest.raises(fa.FaError):  # shifted by one row: neither in place nor apart
        fa.rotary_apply(yq[:, :, :-1], None, freqs, mscale, out=yq[:, :, 1:])


def test_both_parts_of_packed_rows_in_one_call():
    """Queries and keys of one packed row in place, by one call: [B, L, heads, D], and [B, heads, D] (a
    decode step, where the row stride of a single row means nothing)."""
    D, Hq, Hk = 64, 4, 2
    freqs, mscale = fa.rotary_freqs(D)
    for B, L, row in ((2, 5, (Hq + 2 * Hk) * D), (3, 1, D), (1, 1, D)):
        x = randn(B, L, Hq + 2 * Hk, D, dtype=torch.bfloat16)
        q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
        want = fa.rotary(q.contiguous(), k.contiguous(), None, freqs, mscale)
        held = x[:, :, Hq + Hk:].clone()
        st = (L * (Hq + 2 * Hk) * D, D, row)
        assert fa.fa_rotary(q.data_ptr(), k.data_ptr(), q.data_ptr(), k.data_ptr(), [st] * 4, None, 0,
                            freqs.data_ptr(), D, mscale, 0, 0, B, Hq, Hk, L, D, fa.FA_BF16,
                            torch.cuda.current_stream().cuda_stream) == fa.FA_OK
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(x[:, :, Hq + Hk:], held)


@pytest.mark.parametrize("inter,rd", [(False, 128), (True, 64), (False, 24)])
def test_rotary_gradient(inter, rd):
    """The gradient against its formula, against differences, and of broadcast gradients."""
    B, Hq, Hk, L, D = 2, 3, 1, 19, 128
    freqs, mscale = fa.rotary_freqs(rd, scaling="yarn", factor=4.0, original_len=64)
    th, m = thetas(rd, scaling="yarn", factor=4.0, original=64)
    pos = np.repeat(np.arange(5, 5 + L)[None], B, 0).astype(np.int32)
    p = torch.from_numpy(pos).cuda()
    q = randn(B, Hq, L, D, dtype=torch.bfloat16).requires_grad_()
    k = randn(B, Hk, L, D, dtype=torch.bfloat16, seed=1).requires_grad_()
    gq, gk = randn(B, Hq, L, D, dtype=torch.bfloat16, seed=2), randn(B, Hk, L, D, dtype=torch.bfloat16, seed=3)
    qo, ko = fa.rotary(q, k, p, freqs, mscale, inter)
    dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk), retain_graph=True)
    check(dq, gq, pos, th, mscale, inter, inverse=True)
    check(dk, gk, pos, th, mscale, inter, inverse=True)
    # Differences of the definition: the map is linear, so <g, R(x + d) - R(x)> = <R^T g, d>.
    d = np.random.default_rng(0).standard_normal(tuple(q.shape))
    y1, _ = reference(torch.from_numpy(gh.f64(q) + d), pos, th, m, inter)
    y0, _ = reference(q, pos, th, m, inter)
    want = float((gh.f64(gq) * (y1 - y0)).sum())
    have = float((gh.f64(dq) * d).sum())
    # dq is rounded to 8 bits: its error is at most 2^-8 |dq| element by element.
    assert abs(want - have) <= float((np.abs(gh.f64(dq) * d)).sum()) * 2.0 ** -8
    # A sum's gradient is an expanded scalar (strides of 0); an unused output has none.
    (dk2,) = torch.autograd.grad(ko.float().sum(), k)
    check(dk2, torch.ones_like(k), pos, th, mscale, inter, inverse=True)


def test_rotary_second_derivative_and_unused_branches():
    freqs, mscale = fa.rotary_freqs(64)
    q = randn(1, 2, 8, 64, dtype=torch.bfloat16).requires_grad_()
    k = randn(1, 2, 8, 64, dtype=torch.bfloat16, seed=1)
    qo, ko = fa.rotary(q, k, None, freqs, mscale)
    assert not ko.requires_grad or ko.grad_fn is not None
    k2 = randn(1, 3, 8, 64, dtype=torch.bfloat16, seed=5).requires_grad_()
    q2, k2o = fa.rotary(q.detach(), k2, None, freqs, mscale)  # keys alone need a gradient
    g2 = randn(1, 3, 8, 64, dtype=torch.bfloat16, seed=6)
    (dk2,) = torch.autograd.grad((q2, k2o), k2, (torch.ones_like(q2), g2))
    assert torch.equal(dk2, fa.rotary_apply(g2, None, freqs, mscale, inverse=True))
    g = randn(1, 2, 8, 64, dtype=torch.bfloat16, seed=2).requires_grad_()
    (dq,) = torch.autograd.grad(qo, q, g, create_graph=True)
    h = randn(1, 2, 8, 64, dtype=torch.bfloat16, seed=3)
    (dg,) = torch.autograd.grad(dq, g, h)  # dq = R^T g, so the gradient of <h, dq> is R h
    assert torch.equal(dg, fa.rotary_apply(h, None, freqs, mscale))


def test_rotary_infinities_stay_in_their_pair():
    freqs, mscale = fa.rotary_freqs(64)
    x = randn(1, 1, 4, 64, dtype=torch.bfloat16)
    x[0, 0, 1, 5], x[0, 0, 2, 40] = math.inf, math.nan
    y = fa.rotary_apply(x, None, freqs, mscale)
    bad = ~torch.isfinite(y)
    assert set(map(tuple, bad.nonzero().tolist())) <= {(0, 0, 1, 5), (0, 0, 1, 37), (0, 0, 2, 8),
                                                       (0, 0, 2, 40)}
    assert bad[0, 0, 1, 37] and bad[0, 0, 2, 8]


def test_rotary_streams_graph_and_empty():
    freqs, mscale = fa.rotary_freqs(64)
    x = randn(2, 2, 16, 64, dtype=torch.float16)
    want = fa.rotary_apply(x, None, freqs, mscale)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fa.rotary_apply(x, None, freqs, mscale, out=out)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fa.rotary_apply(x, None, freqs, mscale)) and not torch.equal(out, want)
    assert fa.rotary_apply(x[:, :, :0], None, freqs, mscale).shape == (2, 2, 0, 64)
    assert fa.rotary_apply(x[:0], None, freqs, mscale).shape == (0, 2, 16, 64)


def test_rotary_forward_and_backward_in_a_graph():
    """Both directions captured and replayed on new values (no eager graph of the leaves is alive:
    torch refuses such a capture, whatever the operation)."""
    freqs, mscale = fa.rotary_freqs(64)
    q = randn(1, 2, 32, 64, dtype=torch.bfloat16).requires_grad_()
    k = randn(1, 1, 32, 64, dtype=torch.bfloat16, seed=1).requires_grad_()
    gq, gk = randn(1, 2, 32, 64, dtype=torch.bfloat16, seed=2), randn(1, 1, 32, 64, dtype=torch.bfloat16, seed=3)

    def step():
        out = fa.rotary(q, k, None, freqs, mscale)
        return torch.autograd.grad(out, (q, k), (gq, gk))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dq, dk = step()
    gq.mul_(-2.0)
    gk.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dq, fa.rotary_apply(gq, None, freqs, mscale, inverse=True))
    assert torch.equal(dk, fa.rotary_apply(gk, None, freqs, mscale, inverse=True))


def test_rotary_then_attention_depends_on_distances_only():
    """Shifting every position by the same amount leaves attention as it is (relative positions):
    O moves by the 16-bit rounding of the rotated operands alone."""
    B, H, L, D = 1, 2, 160, 64
    q, k, v = (randn(B, H, L, D, dtype=torch.float16, seed=i) for i in range(3))
    freqs, mscale = fa.rotary_freqs(D)
    outs = []
    for shift in (0, 1000000):
        pos = torch.arange(shift, shift + L, dtype=torch.int32, device="cuda")
        outs.append(fa.attention(*fa.rotary(q, k, pos, freqs, mscale), v, causal=True).float())
    # A logit is a sum of 64 products of values rounded to 2^-11: off by at most
    # 2 * 2^-11 * |q||k| / 8 < 2^-10 * 12 * 12 / 8 < 0.02, O by that times the spread of v (< 5).
    assert float((outs[0] - outs[1]).abs().max()) <= 0.1
