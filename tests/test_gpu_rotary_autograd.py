"""rotary as a part of torch's autograd: forward mode, errors in the backward, tensors written in place.

The map is linear, so derivatives are compared bit for bit with the map itself on the derivative's
operand (the same kernel, the same roundings)."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import make_cache, status
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu
B, HQ, HK, L, D = 2, 3, 1, 9, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def operands(dtype=torch.bfloat16):
    freqs, mscale = fa.rotary_freqs(D, scaling="yarn", factor=4.0, original_len=64)
    x = [randn(B, h, L, D, dtype=dtype, seed=i) for i, h in enumerate((HQ, HK, HQ, HK))]
    return (*x, freqs, mscale)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("which", ["q", "k", "both"])
def test_tangents_are_turned(which, inter):
    q, k, tq, tk, freqs, mscale = operands()
    want, want_k = fa.rotary(q, k, None, freqs, mscale, inter)
    with fwd.dual_level():
        dq = fwd.make_dual(q, tq) if which != "k" else q
        dk = fwd.make_dual(k, tk) if which != "q" else k
        out = fa.rotary(dq, dk, None, freqs, mscale, inter)
        for o, value, t, has in zip(out, (want, want_k), (tq, tk), (which != "k", which != "q")):
            primal, tangent = fwd.unpack_dual(o)
            assert torch.equal(primal, value)
            assert (tangent is not None) == has
            if has:
                assert torch.equal(tangent, fa.rotary_apply(t, None, freqs, mscale, inter))


def test_broadcast_and_differentiable_tangents():
    """A tangent with strides of 0, and one that needs a gradient itself (forward over reverse)."""
    q, k, tq, _, freqs, mscale = operands(torch.float16)
    q.requires_grad_()
    t = tq[:, :1].clone().requires_grad_()
    g = randn(B, HQ, L, D, dtype=torch.float16, seed=7)
    back = fa.rotary_apply(g, None, freqs, mscale, inverse=True)
    with fwd.dual_level():
        out, _ = fa.rotary(fwd.make_dual(q, t.expand(B, HQ, L, D)), k, None, freqs, mscale)
        primal, tangent = fwd.unpack_dual(out)
        full = t.detach().expand(B, HQ, L, D).contiguous()
        assert torch.equal(tangent.detach(), fa.rotary_apply(full, None, freqs, mscale))
        dt, = torch.autograd.grad(tangent, t, g, retain_graph=True)
        assert torch.equal(dt, back.sum(1, keepdim=True))
        dq, = torch.autograd.grad(primal, q, g)
        assert torch.equal(dq, back)


def test_writes_are_seen_by_autograd():
    """Every call that writes a caller's tensor raises its version, so that a backward which saved the
    old values is refused; tensors of inference mode, which have no version, can be written too."""
    q, k, x, _, freqs, mscale = operands()
    w = torch.ones_like(x, requires_grad=True)
    y = (w * x).sum()  # saves x
    fa.rotary_apply(x, None, freqs, mscale, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    for quant in (False, True):
        kc, vc, ke, ve = make_cache(B, HK, D, q.dtype, quant)
        bt = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
        sl = torch.full((B,), L, dtype=torch.int32, device="cuda")
        dense = tuple(torch.empty_like(k) for _ in range(2))
        row = q[:, :, 0].contiguous()
        o, lse = torch.empty_like(row), torch.empty((B, HQ), device="cuda")
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        calls = [((kc, vc, ke, ve), lambda: fa.cache_append(k, k, kc, vc, bt, sl, k_exp=ke, v_exp=ve)),
                 (dense, lambda: fa.cache_read(kc, vc, bt, sl, L, k_exp=ke, v_exp=ve, out=dense)),
                 ((o, lse, ws), lambda: fa.decode_paged(row, kc, vc, bt, sl, out=o, lse=lse, workspace=ws,
                                                        k_exp=ke, v_exp=ve))]
        if not quant:
            calls.append(((o, lse, ws), lambda: fa.decode_shared_prefix(
                row, kc, vc, bt[0], 1, bt, sl, out=o, lse=lse, workspace=ws)))
            one, one_lse = o[:, :1].contiguous(), lse[:, :1].contiguous()
            calls.append(((one, one_lse, ws), lambda: fa.decode_paged(
                row[:, :1].contiguous(), kc, vc, bt, sl, out=one, lse=one_lse, workspace=ws)))
        for tensors, call in calls:
            tensors = [t for t in tensors if t is not None]
            before = [t._version for t in tensors]
            call()
            assert all(t._version > v for t, v in zip(tensors, before))
    with torch.inference_mode():
        z = x.clone()
    assert torch.equal(fa.rotary_apply(z, None, freqs, mscale, out=z), fa.rotary_apply(x, None, freqs, mscale))
    assert status() == fa.FA_OK
