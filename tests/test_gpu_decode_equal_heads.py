"""decode_paged with as many cache heads as query heads (the kernel of fa_decode_paged) over caches
that cache_append wrote, against the definition in 64 bits; tolerances as in test_gpu_decode_gqa.py."""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import make_cache, status
from test_gpu_decode_gqa import check, fill
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def test_refusals_before_anything_is_read():
    """A cache whose bytes are not rows of q's type, outputs and workspaces that are too small."""
    D, H, B = 64, 2, 3
    q = randn(B, H, D, dtype=torch.bfloat16)
    kc, vc, _, _ = make_cache(2, H, D, torch.bfloat16, False)
    bt = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    sl = torch.ones(B, dtype=torch.int32, device="cuda")
    k8, v8, ke, ve = make_cache(2, H, D, torch.bfloat16, True)
    launched = fa.fa_launch_count()
    with pytest.raises(TypeError):
        fa.decode_paged(q, k8, v8, bt, sl)  # e4m3 rows without their exponents: half the bytes
    with pytest.raises(TypeError):
        fa.decode_paged(q, kc.half(), vc.half(), bt, sl)
    with pytest.raises(TypeError):
        fa.decode_paged(q, kc, vc.half(), bt, sl)
    with pytest.raises(TypeError):
        fa.decode_paged(q, kc, vc, bt.long(), sl)
    for bad in (dict(out=torch.empty(B, H, D // 2, device="cuda", dtype=q.dtype)),
                dict(out=torch.empty(B, H, D, device="cuda", dtype=torch.float16)),
                dict(out=torch.empty(B, H, D, dtype=q.dtype)),
                dict(lse=torch.empty(B, H - 1, device="cuda")),
                dict(lse=torch.empty(B, H, device="cuda", dtype=torch.float64)),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fa.decode_paged(q, kc, vc, bt, sl, **bad)
    for args in ((q, kc[:, :, :8].contiguous(), vc[:, :, :8].contiguous(), bt, sl),
                 (q, kc, vc[:1], bt, sl), (q, kc, vc, bt[:1], sl), (q, kc, vc, bt, sl[:1]),
                 (q, kc, vc, bt.cpu(), sl), (q, kc.transpose(2, 3), vc, bt, sl),
                 (q[:, :, :32].contiguous(), kc, vc, bt, sl)):
        with pytest.raises(ValueError):
            fa.decode_paged(*args)
    with pytest.raises(fa.FaError):
        fa.decode_paged(q, kc, vc, bt, sl, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert fa.fa_launch_count() == launched and status() == fa.FA_OK


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16), (64, torch.bfloat16),
                                     (128, torch.float16)], ids=str)
@pytest.mark.parametrize("lens,H", [([0, 1, 15, 16, 17, 63, 64, 129, 300, 1000], 3), ([1], 1), ([3000], 2),
                                    ([17, 2001, 0], 4), ([5] * 700, 1)],
                         ids=["mixed", "one", "long", "split", "many"])
def test_unused_slots_may_hold_anything(D, dtype, lens, H):
    """Pages that cache_append wrote in part, all other slots NaN: one CTA per row and split rows."""
    rng = np.random.default_rng(D + len(lens))
    kc, vc, _, _, bt, sl, ks, vs = fill(rng, lens, H, D, dtype, False)
    q = randn(len(lens), H, D, dtype=dtype, seed=H)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)
    for c in (kc, vc):  # infinities there instead
        c.nan_to_num_(math.inf)
    o2, lse2 = fa.decode_paged(q, kc, vc, bt, sl)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
