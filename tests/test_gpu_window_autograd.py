"""attention_window as a part of torch's autograd: what it refuses, and that forward and backward belong together."""
import math

import pytest
import torch
import torch.autograd.forward_ad as fwd

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_window import operands, status
from window_reference import reference, sees

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_mode_is_refused(which):
    x = list(operands(1, 1, 4, 2, 64, 64, 64, BF16)[:3])
    with fwd.dual_level():
        x[which] = fwd.make_dual(x[which], torch.ones_like(x[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            fa.attention_window(*x, 8)
        x[which] = x[which].requires_grad_()
        with pytest.raises(NotImplementedError, match="forward-mode"):
            fa.attention_window(*x, 8)
    assert status() == fa.FA_OK


@pytest.mark.parametrize("which", [0, 1, 2])
def test_function_transforms_are_refused(which):
    """Errors, whichever operand is transformed, and nothing launched."""
    x = list(operands(2, 2, 4, 2, 64, 64, 64, FP16)[:3])

    def f(y, forward=fa.attention_window):
        a = x[:which] + [y] + x[which + 1:]
        return forward(*a, 8, 1)

    launched = fa.fa_launch_count()
    for call in (lambda: torch.func.grad(lambda y: f(y).float().sum())(x[which]),
                 lambda: torch.func.vjp(f, x[which]),
                 lambda: torch.func.jvp(f, (x[which],), (x[which],)),
                 lambda: torch.vmap(f)(torch.stack([x[which]] * 3)),
                 lambda: torch.vmap(lambda y: f(y, fa.window_forward))(torch.stack([x[which]] * 3))):
        with pytest.raises(RuntimeError):  # (NotImplementedError is one)
            call()
    assert fa.fa_launch_count() == launched and status() == fa.FA_OK


def test_gradients_of_some_operands():
    """Of the three only what asks for one gets a gradient, the same as when all do."""
    q, k, v, do = operands(3, 2, 4, 2, 200, 200, 64, BF16)
    every = [x.detach().requires_grad_() for x in (q, k, v)]
    want = torch.autograd.grad(fa.attention_window(*every, 30, 2), every, do)
    for which in range(3):
        x = [y.detach() for y in (q, k, v)]
        x[which].requires_grad_()
        fa.attention_window(*x, 30, 2).backward(do)
        assert torch.equal(x[which].grad, want[which])
        assert all(y.grad is None for i, y in enumerate(x) if i != which)


@pytest.mark.parametrize("Hq,Hk,Lq,Lk,D,window,sinks", [
    (4, 2, 200, 200, 64, 50, 4), (3, 1, 300, 300, 128, 5000, 0), (2, 2, 150, 400, 64, 100, 130), (4, 4, 400, 150, 64, 20, 1)])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_the_backward_is_the_slope_of_the_forward(which, Hq, Hk, Lq, Lk, D, window, sinks):
    """f = sum(o do) from window_forward on both sides of the operands, along the gradient that window_backward
    gives: (f(x + s) - f(x - s)) / 2 is the sum of gradient times step, and terms of third order and up.

    Tolerance.  Operands are multiples of 2^-5, the step of 2^-4 and half of it of 2^-5, all below 8: exact in fp16.
    Each o is off by its bound e of window_reference at most, a difference by sum |do| (e+ + e-) / 2.  With c3 and c5
    the terms of third and fifth order of the whole step, the half step gives d/2 + c3/8 + c5/32, so that
    (8 half - whole) / 3 = d - c5/4; at an rms step of a quarter (scores move by about a quarter) c5 is below c3.
    The gradient is off by its bound in window_reference.  The step runs along the gradient, so that the slope is a
    sum of squares; where the bounds together pass a quarter of it the case would show little, and fails."""
    dtype, scale, G = FP16, 1 / math.sqrt(D), Hq // Hk
    q, k, v, do = operands(4, 1, Hq, Hk, Lq, Lk, D, dtype)
    x = dict(zip("qkv", ((y.float() * 32).round().clamp(-192, 192).div(32).to(dtype) for y in (q, k, v))))
    o, lse = fa.window_forward(x["q"], x["k"], x["v"], window, sinks)
    grads = fa.window_backward(x["q"], x["k"], x["v"], o, lse, do, window, sinks)
    grad = dict(zip("qkv", grads))[which].double()
    mask = sees(Lq, Lk, window, sinks)

    def refs(a, do_=None):
        return [reference(a["q"][0, h * G:h * G + G], a["k"][0, h], a["v"][0, h], mask, scale,
                          None if do_ is None else do_[0, h * G:h * G + G]) for h in range(Hk)]

    bound_grad = torch.stack([r["d" + which][1] for r in refs(x, do)]).reshape(grad.shape)
    step = (grad * (0.25 / float(grad.square().mean().sqrt())) * 16).round().clamp(-24, 24) / 16

    def f(h):
        a = {**x, which: (x[which].double() + h * step).to(dtype)}
        assert torch.equal(a[which].double(), x[which].double() + h * step)
        out = fa.window_forward(a["q"], a["k"], a["v"], window, sinks)[0].double()
        off = sum(float((do[0, i * G:i * G + G].double().abs() * r["o"][1]).sum()) for i, r in enumerate(refs(a)))
        return float((out * do.double()).sum()), off

    (a, ea), (b, eb), (c, ec), (d, ed) = f(1.0), f(-1.0), f(0.5), f(-0.5)
    assert status() == fa.FA_OK
    whole, half = (a - b) / 2, (c - d) / 2
    third = (whole - 2 * half) * 4 / 3
    got, want = (8 * half - whole) / 3, float((grad * step).sum())
    bound = (8 * (ec + ed) / 2 + (ea + eb) / 2) / 3 + abs(third) / 4 + float((bound_grad * step.abs()).sum())
    assert bound <= want / 4, (bound, want)
    assert abs(got - want) <= bound, (got, want, bound)
