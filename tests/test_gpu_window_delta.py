"""Rows of few keys take Delta = rowsum(dO o O) from P and dP in fp32 instead of from the rounded O (fa_window_bwd.cu).

What that is worth shows in the gradients' errors against 64 bits, as a multiple of what rounding the exact gradients
to 16 bits costs (root mean squares; element by element either form stays within the bounds of window_reference).
dS is rounded to 16 bits before the products, dQ_i = sum_j dS_ij K_j once more behind them.  Roundings are
independent and relative, so that both have the same relative mean square: with dS's alone the ratio is
sqrt(2) = 1.41 (fp32's part is 2^-13 of that).  A Delta from the rounded O is off by dO's product with O's rounding, the
same for all keys of the row: 1.7 to 1.8 at 8 keys.  Both forms are restated below in 64 bits; the limit of a tile lies
half way between the two, which have to be a tenth apart there."""
import math

import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_window import operands, status
from window_reference import sees

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def rms(x):
    return float(x.square().mean().sqrt())


def restated(q, k, v, do, mask, scale, rounded_o):
    """dQ and dK [Hq or Hk, L, D] in 64 bits from P and dS rounded to the operands' type, with Delta from the rounded O or
    exact; and the exact ones."""
    dt, G = q.dtype, q.shape[0] // k.shape[0]
    q, do = (x.double().unflatten(0, (-1, G)) for x in (q, do))
    k, v = k.double()[:, None], v.double()[:, None]
    y = torch.where(mask, q @ k.mT * scale, -math.inf)
    p = torch.where(mask, torch.softmax(y, -1), 0.0).nan_to_num(0.0)
    dp = do @ v.mT
    o = (p.to(dt).double() @ v).to(dt).double() if rounded_o else p @ v
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    exact = p * (dp - (p * dp).sum(-1, keepdim=True))
    ds = ds.to(dt).double()
    return [(t(ds), t(exact)) for t in (lambda s: (s @ k * scale).flatten(0, 1),
                                        lambda s: (s.mT @ q * scale).sum(1))]


# B = 1; rows (of dQ) and keys (of dK) that are compared, tile by tile where every row has few keys
CASES = [
    (8, 2, 1000, 1000, 64, BF16, 8, 0, "tiles"),      # a short window: every tile, the last one ragged
    (8, 8, 700, 900, 64, BF16, 8, 0, "tiles"),        # behind earlier keys
    (8, 4, 900, 700, 64, FP16, 8, 0, "tiles"),        # rows without a key in front, 72 of the first tile that has any
    (8, 2, 560, 560, 128, BF16, 6, 2, "tiles"),
    (16, 4, 700, 700, 64, BF16, 700, 0, (0, 24)),     # a long one: the first rows
    (16, 4, 900, 700, 64, BF16, 600, 0, (200, 224)),  # ... which stand behind 200 without a key
]


@pytest.mark.parametrize("Hq,Hk,Lq,Lk,D,dtype,window,sinks,rows", CASES)
def test_error_of_rows_of_few_keys(Hq, Hk, Lq, Lk, D, dtype, window, sinks, rows):
    q, k, v, do = operands(1, 1, Hq, Hk, Lq, Lk, D, dtype)
    scale = 1 / math.sqrt(D)
    o, lse = fa.window_forward(q, k, v, window, sinks)
    dq, dk, _ = fa.window_backward(q, k, v, o, lse, do, window, sinks)
    assert status() == fa.FA_OK
    mask = sees(Lq, Lk, window, sinks)
    pre, mine = (restated(q[0], k[0], v[0], do[0], mask, scale, r) for r in (True, False))
    for name, got, before, now, L in (("dq", dq, pre[0], mine[0], Lq), ("dk", dk, pre[1], mine[1], Lk)):
        exact = now[1]
        parts = [(t, min(t + 128, L)) for t in range(0, L, 128)] if rows == "tiles" else \
            [rows] if name == "dq" else []
        for a, b in parts:
            want = exact[:, a:b]
            if b - a < (32 if rows == "tiles" else 1) or not want.any():  # (too few to tell)
                continue
            alone = rms(want.to(dtype).double() - want)

            def ratio(x):
                return rms(x[:, a:b].double() - want) / alone

            rounded, summed = (ratio(x[0].to(dtype)) for x in (before, now))
            assert rounded > 1.1 * summed, (name, a, rounded, summed)
            assert ratio(got[0]) <= (rounded + summed) / 2, (name, a, ratio(got[0]), rounded, summed)
