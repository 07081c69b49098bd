"""Calls of the sliding-window and chunk operators that other tests leave out: captured through autograd, into parts of one
packed tensor, over very many heads, on several streams at once, on tensors of inference mode."""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_decode_gqa import fill
from test_gpu_rotary import randn
from test_gpu_window import check, operands, run, status

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def test_forward_and_gradients_captured_through_autograd():
    q, k, v, do = operands(1, 2, 4, 2, 500, 500, 64, BF16)
    static = [x.clone().requires_grad_() for x in (q, k, v)]

    def step():
        o = fa.attention_window(*static, 60, 5)
        return o.detach(), torch.autograd.grad(o, static, do)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, grads = step()
    for seed in (2, 3):
        new = operands(seed, 2, 4, 2, 500, 500, 64, BF16)
        with torch.no_grad():
            for x, y in zip((*static, do), new):
                x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = run(*new, 60, 5)
        assert torch.equal(o, want["o"])
        assert all(torch.equal(a, want[n]) for a, n in zip(grads, ("dq", "dk", "dv")))


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 3)])
def test_outputs_as_parts_of_packed_tensors(Hq, Hk):
    """q, k, v and o in one tensor [B, L, heads, D], the gradients in another."""
    B, L, D, H = 2, 300, 64, 2 * Hq + 2 * Hk
    parts = [slice(0, Hq), slice(Hq, Hq + Hk), slice(Hq + Hk, Hq + 2 * Hk), slice(Hq + 2 * Hk, H)]
    x = randn(B, L, H, D, dtype=FP16, seed=4).transpose(1, 2)
    q, k, v, o = (x[:, p] for p in parts)
    do = randn(B, L, Hq, D, dtype=FP16, seed=5).transpose(1, 2)
    plain = run(*(y.clone() for y in (q, k, v)), do, 70, 3)
    g = torch.full((B, L, H, D), math.nan, device="cuda", dtype=FP16).transpose(1, 2)
    _, lse = fa.window_forward(q, k, v, 70, 3, out=o)
    grads = [g[:, p] for p in parts[:3]]
    fa.window_backward(q, k, v, o, lse, do, 70, 3, grads=grads)
    assert status() == fa.FA_OK
    assert torch.equal(o, plain["o"]) and torch.equal(lse, plain["lse"])
    assert all(torch.equal(a, plain[n]) for a, n in zip(grads, ("dq", "dk", "dv")))
    assert g[:, parts[3]].isnan().all()


def test_more_heads_than_a_grid_dimension_takes():
    q, k, v, do = operands(6, 70000, 2, 1, 3, 4, 64, FP16)
    out = run(q, k, v, do, 2, 1)
    for b in (0, 1, 32767, 32768, 65535, 65536, 69999):
        one = slice(b, b + 1)
        check({n: t[one] for n, t in out.items()}, q[one], k[one], v[one], do[one], 2, 1, 1 / 8)
    # The same rows whatever stands beside them.
    part = slice(69000, 70000)
    again = run(*(x[part].contiguous() for x in (q, k, v, do)), 2, 1)
    assert all(torch.equal(out[n][part], again[n]) for n in again)


def test_several_streams_at_once():
    """Calls that overlap, each with outputs and workspaces of its own, give the bits of calls alone."""
    rng = np.random.default_rng(7)
    kc, vc, ke, ve, bt, sl, _, _ = fill(rng, [900, 40, 3000], 2, 64, FP16, True)
    lens = torch.tensor([40, 40, 40], dtype=torch.int32, device="cuda")
    x = operands(8, 1, 4, 2, 900, 900, 64, FP16)
    chunk, few, row = randn(3, 4, 40, 64, dtype=FP16), randn(3, 4, 3, 64, dtype=FP16), randn(3, 4, 64, dtype=FP16)
    kw = dict(k_exp=ke, v_exp=ve)

    def backward():
        o, lse = fa.window_forward(*x[:3], 100, 9)
        return (o, lse, *fa.window_backward(*x[:3], o, lse, x[3], 100, 9))

    calls = [backward, lambda: fa.attention_paged(chunk, kc, vc, bt, sl, lens, **kw),
             lambda: fa.attention_paged(few, kc, vc, bt, sl, **kw),
             lambda: fa.decode_paged(row, kc, vc, bt, sl, window=200, sinks=3, **kw)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(20):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(c())
    torch.cuda.synchronize()
    assert status() == fa.FA_OK
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i % len(calls)])), i % len(calls)


def test_tensors_of_inference_mode():
    q, k, v, do = operands(9, 1, 4, 2, 200, 200, 64, BF16)
    want = run(q, k, v, do, 30, 2)
    with torch.inference_mode():
        a = [y.clone() for y in (q, k, v)]
        out = torch.empty_like(a[0])
        assert torch.equal(fa.attention_window(*a, 30, 2), want["o"])
        fa.window_forward(*a, 30, 2, out=out)
        assert torch.equal(out, want["o"])


def test_very_many_sequences_with_few_new_tokens():
    """More launches than one, against single tokens of the same sequences."""
    B = 20000
    rng = np.random.default_rng(10)
    kc, vc, _, _, _, _, _, _ = fill(rng, [640], 1, 64, BF16, False)
    pages = kc.shape[0]
    bt = torch.randint(0, pages, (B, 3), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    sl = torch.randint(0, 49, (B,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    q = randn(B, 2, 2, 64, dtype=BF16)
    nl = (sl > 0).int()
    o, lse = fa.attention_paged(q, kc, vc, bt, sl, nl)
    od, lsed = fa.decode_paged(q[:, :, 0].contiguous(), kc, vc, bt, sl)
    assert status() == fa.FA_OK
    assert not o[:, :, 1].any() and (lse[:, :, 1] == -math.inf).all()
    # Some tables name pages that belong to nobody and hold NaN: rows that see one are NaN, no others.
    nobody = kc.float().isnan().flatten(1).any(1)
    seen = torch.arange(3, device="cuda")[None] * 16 < sl[:, None]
    lost = (nobody[bt.long()] & seen).any(1)
    assert torch.equal(o[:, :, 0].isnan(), lost[:, None, None].expand(B, 2, 64))
    assert torch.equal(od.isnan(), lost[:, None, None].expand(B, 2, 64))
    # Each is off by eps/2 of A = sum p |v| <= max |v| (P) and eps/2 of itself (O), and by 2^-14 of A for the sums of up
    # to 64 products in fp32 and the exponentials; they differ by twice that at most.
    eps, kept = torch.finfo(BF16).eps, ~lost
    top = float(vc.float().nan_to_num(0.0).abs().max())
    a, b = o[kept][:, :, 0].double(), od[kept].double()
    assert ((a - b).abs() <= (eps + 2.0 ** -13) * top + eps * torch.maximum(a.abs(), b.abs())).all()
    some = (sl > 0) & kept
    assert ((lse[some][:, :, 0] - lsed[some]).abs() <= 2.0 ** -16 * (1 + lsed[some].abs())).all()
