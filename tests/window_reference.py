"""Attention under a sliding window in 64 bits, and how far 16-bit kernels with fp32 sums may be off.

With weights p_j (softmax) and A = sum_j p_j |v_j|, element by element:
* a score is a sum of D exact products in fp32, off by at most D 2^-23 sum_i |q_i k_i| |scale| (an addition
  is off by 2^-23 where the tensor core cuts instead of rounding); d is the largest such error over the
  row's keys, plus 2^-20 for the exponentials (2^-22 each), the shift by the reference and the row's sum;
  it changes a weight by a factor within 1 + 2d and its share by twice that;
* P is rounded to 16 bits, half a step: eps/2 of each weight, or below fp16's normal range 2^-25 of the
  row's largest weight (the kernels' reference lies at most 2^8 below the largest score, so that the
  weights in units of the reference are at least those in units of the largest); a weight below 2^-126
  may be lost, whatever the type (the exponential gives zero there), and with it 2^-126 of its factor;
* a sum of n products is off by at most n 2^-23 of the sum of magnitudes;
* O is rounded once: eps/2 |O| (and 2^-25 in fp16).
Gradients, from the same P (now exp(score - LSE) with LSE in fp32: 2^-24 |LSE| more in d):
* dP is a sum of D products; Delta = rowsum(dO o O) from the rounded O: off by sum |dO| err(O) and its sum;
* dS = P o (dP - Delta) is rounded to 16 bits, like P, before the products with Q and K;
* each gradient is rounded once.
"""
import math

import torch

U = 2.0 ** -23


def sees(Lq, Lk, window, sinks, device="cuda"):
    t = torch.arange(Lq, device=device)[:, None] + (Lk - Lq)
    j = torch.arange(Lk, device=device)[None]
    return (j <= t) & ((j > t - window) | (j < sinks))


def reference(q, k, v, mask, scale, do=None):
    """One group: q [G, Lq, D], k, v [Lk, D], do like q, in any type; mask [Lq, Lk].  Returns a dict of
    (value, bound) in 64 bits: o, lse and, with do, dq, dk, dv."""
    dt = q.dtype
    eps, tiny = torch.finfo(dt).eps, 2.0 ** -25 if dt == torch.float16 else 2.0 ** -126
    q, k, v = q.double(), k.double(), v.double()
    D, n = q.shape[-1], mask.shape[-1]
    y = (q @ k.mT) * scale
    ey = (q.abs() @ k.abs().mT) * (abs(scale) * D * U)
    y, ey = torch.where(mask, y, -math.inf), torch.where(mask, ey, 0.0)
    some = mask.any(-1)
    lse = torch.logsumexp(y, -1)
    p = torch.where(mask, torch.exp(y - torch.where(some, lse, 0.0)[..., None]), 0.0)
    d = ey.amax(-1, keepdim=True) + 2.0 ** -20
    A = p @ v.abs()
    top = p.amax(-1, keepdim=True)
    o = p @ v
    eo = (eps / 2 + 4 * d + n * U) * A + n * tiny * top * v.abs().amax() + eps / 2 * o.abs() + tiny
    out = {"o": (o, eo), "lse": (lse, d[..., 0] + 2.0 ** -22 * (1 + torch.where(some, lse, 0.0).abs()))}
    if do is None:
        return out
    do = do.double()
    d = d + 2.0 ** -22 * (1 + torch.where(some, lse, 0.0).abs()[..., None])
    dp = do @ v.mT
    delta = (do * o).sum(-1, keepdim=True)
    edp = (do.abs() @ v.abs().mT) * (D * U)
    edelta = (do.abs() * eo).sum(-1, keepdim=True) + D * U * (do.abs() * o.abs()).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    eds = (2 * d + eps / 2) * ds.abs() + (1 + 2 * d) * p * (edp + edelta) + \
        torch.where(mask, tiny * (1 + (dp - delta).abs()), 0.0)
    ep = (2 * d + eps / 2) * p + torch.where(mask, tiny, 0.0)
    s = abs(scale)
    G = q.shape[0]

    def rounded(x, e):
        return x, e + eps / 2 * x.abs() + tiny

    out["dq"] = rounded(ds @ k * scale, s * ((eds + n * U * ds.abs()) @ k.abs()))
    rows = G * q.shape[1]
    out["dk"] = rounded((ds.mT @ q).sum(0) * scale, s * ((eds + rows * U * ds.abs()).mT @ q.abs()).sum(0))
    out["dv"] = rounded((p.mT @ do).sum(0), ((ep + rows * U * p).mT @ do.abs()).sum(0))
    return out


def within(got, value_bound, what):
    value, bound = value_bound
    got = got.double()
    same = (got == value)  # (infinities)
    off = torch.where(same, 0.0, (got - value).abs())
    bad = ~(off <= bound)  # (a NaN is bad)
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {float(got[i])}, "
                             f"expected {float(value[i])} within {float(bound[i])}")
