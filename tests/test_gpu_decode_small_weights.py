"""Many small weights behind a large one (a key that every query attends to, as the first token of a
text often is) over fp16 and e4m3 caches, where P is rounded to fp16.

One key has score 0, all others -20.5 bits.  Half of an output row's elements come from the one key alone,
half from the others alone, so that what the others lose is not hidden behind it.

Tolerance.  With the largest weight of a running reference at 2^7 or more, the others are 2^-13.5 and more:
normal in fp16, each off by eps/2 at most, where a reference of 1 would leave them 4 bits (2^-20.5 is
11.3 steps of 2^-24: off by 2.8%).  The sums are fp32 and the exponentials good to 2^-22, 2^-20 in
all; O is rounded once, eps/2."""
import math

import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import PAGE, make_cache, status

pytestmark = pytest.mark.gpu
BITS = 20.5
D = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def sequence(n, Hk, q8, at):
    """One sequence of n tokens; the large key is token `at`."""
    pages = -(-n // PAGE)
    kc, vc, ke, ve = make_cache(pages, Hk, D, torch.float16, q8)
    k = torch.zeros((1, Hk, n, D), device="cuda", dtype=torch.float16)
    v = torch.zeros_like(k)
    k[:, :, at, 0] = 1.0
    v[:, :, :, D // 2:] = 1.0
    v[:, :, at, :D // 2], v[:, :, at, D // 2:] = 1.0, 0.0
    bt = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    fa.cache_append(k, v, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    return kc, vc, ke, ve, bt, sl


def check(o, n):
    w = 2.0 ** -BITS
    want = torch.tensor([1.0 / (1.0 + (n - 1) * w), (n - 1) * w / (1.0 + (n - 1) * w)], dtype=torch.float64)
    got = o.double().cpu().unflatten(-1, (2, D // 2))
    err = (got / want[:, None] - 1.0).abs()
    eps = torch.finfo(torch.float16).eps
    assert float(err.max()) <= eps * (1 + 2.0 ** -8) + 2.0 ** -19, float(err.max())


@pytest.mark.parametrize("q8", [True, False], ids=["e4m3", "fp16"])
@pytest.mark.parametrize("B,Hk,group,at", [(700, 8, 1, 0), (320, 8, 12, 0), (700, 8, 4, 900), (1, 1, 1, 0), (3, 2, 2, 5)])
def test_grouped_decode(q8, B, Hk, group, at):
    """Every sequence of the batch is the same one."""
    n = 1000
    kc, vc, ke, ve, bt, sl = sequence(n, Hk, q8, at)
    q = torch.zeros((B, Hk * group, D), device="cuda", dtype=torch.float16)
    q[:, :, 0] = 1.0
    o, _ = fa._decode_paged_ex(q, kc, vc, bt.repeat(B, 1), sl.repeat(B), BITS * math.log(2.0), k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, n)


@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("at", [0, 2100])
def test_shared_prefix(scale, at):
    n, B, Hk = 4096, 256, 32
    kc, vc, _, _, bt, _ = sequence(n, Hk, False, at)
    q = torch.zeros((B, Hk, D), device="cuda", dtype=torch.float16)
    q[:, :, 0] = scale
    none = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    o, _ = fa.decode_shared_prefix(q, kc, vc, bt[0], n, none, torch.zeros(B, dtype=torch.int32, device="cuda"),
                                   scale * BITS * math.log(2.0))
    assert status() == fa.FA_OK
    check(o, n)
