"""Many small weights behind a large one under a sliding window in fp16, where P is rounded to fp16 for the
contraction: a first token that stays visible often carries nearly all of a row.

One key has score 0, all others -20.5 bits.  Half of an output row's elements come from the one key alone, half
from the others alone, so that what the others lose is not hidden behind it.

Tolerance.  With the largest weight of a running reference at 2^7 or more, the others are 2^-13.5 and more:
normal in fp16, each off by eps/2 at most, where a reference of 1 would leave them 4 bits (2^-20.5 is
11.3 steps of 2^-24: off by 2.8%).  A sum of n products and one of n weights are off by n 2^-23 each.  The score of
20.5 bits is off by three roundings of 2^-24 (scale, scale times log2 e, their product), 2^-18.6 of a weight, the
exponentials and the normalisation by 2^-20: 2^-18 in all.  O is rounded once, eps/2, or 2^-25 below fp16's normal
range (rows of few keys: 2^-20.5 a key is under 2^-14 up to 90 keys, where fp16's step is 2^-24).  LSE, up to 21.2, adds three
roundings of 2^-24 and a logarithm's 2^-22 to the score's error: 2^-17."""
import math

import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa

pytestmark = pytest.mark.gpu
BITS = 20.5
FP16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


# at: the large key.
@pytest.mark.parametrize("Hq,Hk,Lq,Lk,D,window,at", [
    (4, 2, 700, 700, 64, 300, 0),        # the first token, single tiles
    (2, 1, 300, 900, 128, 300, 0),       # rows behind earlier keys
    (64, 32, 1000, 1000, 128, 256, 0),   # two heads at a time
    (33, 33, 1500, 1500, 64, 640, 0),    # two tiles of a head at a time
    (2, 2, 700, 700, 128, 5000, 600),    # a key that rows meet late: the reference is raised
])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_small_weights_keep_their_bits(Hq, Hk, Lq, Lk, D, window, at, sign):
    q = torch.zeros((1, Hq, Lq, D), device="cuda", dtype=FP16)
    k = torch.zeros((1, Hk, Lk, D), device="cuda", dtype=FP16)
    v = torch.zeros_like(k)
    q[..., 0] = sign
    k[:, :, at, 0] = 1.0
    v[..., D // 2:] = 1.0
    v[:, :, at, :D // 2], v[:, :, at, D // 2:] = 1.0, 0.0
    o, lse = fa.window_forward(q, k, v, window, 1, sign * BITS * math.log(2.0))
    assert fa.fa_get_device_status(torch.cuda.current_stream().cuda_stream) == fa.FA_OK
    t = torch.arange(Lq, dtype=torch.float64, device="cuda") + (Lk - Lq)
    n = torch.minimum(t + 1, t.new_tensor(float(window))) + ((t >= window) if at == 0 else 0)  # keys that a row sees
    large = ((t >= at) & ((t - window < at) | (at == 0))).double()
    w = 2.0 ** -BITS
    total = large + (n - large) * w
    want = torch.stack((large / total, (n - large) * w / total), -1)
    got = o[0].double().unflatten(-1, (2, D // 2))
    eps = torch.finfo(FP16).eps
    bound = want * (eps * (1 + 2.0 ** -8) + 2.0 ** -18 + 2 * n[:, None] * 2.0 ** -23) + 2.0 ** -25
    err = (got - want[None, :, :, None]).abs().amax((0, 3))
    worst = (err / want.clamp(min=1e-30)).amax()
    assert bool((err <= bound).all()), float(worst)
    assert ((lse[0].double() - (torch.log(total) + BITS * math.log(2.0))).abs() <= 2.0 ** -17).all()
