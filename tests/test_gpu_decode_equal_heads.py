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


@pytest.mark.parametrize("lens,at", [([40, 40, 1], (1, 35)), ([40, 1, 40], (1, 0)), ([16, 2000, 5], (1, 999)),
                                     ([4, 3000, 4], (1, 0)), ([4, 1, 3000], (1, 0))], ids=str)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_key_makes_its_row_nan(lens, at, bad):
    """A NaN score is in every weight of its row: O and LSE are NaN, even where it is the row's only
    score, or a warp's or a split's; as in the kernel of grouped heads.  Other rows keep their bits."""
    D, H, dtype = 64, 2, torch.bfloat16
    rng = np.random.default_rng(len(lens))
    kc, vc, _, _, bt, sl, _, _ = fill(rng, lens, H, D, dtype, False)
    q = randn(len(lens), H, D, dtype=dtype)
    q[:, :, 7] = 1.0  # (an infinity is a score of +inf: inf - inf in every weight)
    good, good_lse = fa.decode_paged(q, kc, vc, bt, sl)
    b, t = at
    kc[int(bt[b, t // 16]), 1, t % 16, 7] = bad
    o, lse = fa.decode_paged(q, kc, vc, bt, sl)
    o2, lse2 = fa._decode_paged_ex(q, kc, vc, bt, sl)
    assert status() == fa.FA_OK
    for x, l in ((o, lse), (o2, lse2)):
        assert torch.isnan(x[b, 1]).all() and torch.isnan(l[b, 1])
    keep = torch.ones(len(lens), H, dtype=torch.bool)
    keep[b, 1] = False
    assert torch.equal(o[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])


@pytest.mark.parametrize("n", [1, 40, 3000])
def test_scores_of_minus_infinity_weigh_nothing(n):
    """Scores of -inf beside finite ones count for nothing; alone they leave O = 0, LSE = -inf, as a row
    without a key."""
    D, dtype = 64, torch.bfloat16
    rng = np.random.default_rng(n)
    kc, vc, _, _, bt, sl, ks, vs = fill(rng, [n, n], 1, D, dtype, False)
    q = randn(2, 1, D, dtype=dtype)
    q[:, :, 0] = 1.0
    table = bt.long()
    for t in range(n):
        if t != 20:  # (sequence 1 keeps one finite score, where it is long enough)
            kc[table[1, t // 16], 0, t % 16, 0] = -math.inf
        kc[table[0, t // 16], 0, t % 16, 0] = -math.inf
    o, lse = fa.decode_paged(q, kc, vc, bt, sl)
    assert status() == fa.FA_OK
    assert not o[0].any() and lse[0, 0] == -math.inf
    if n <= 20:
        assert not o[1].any() and lse[1, 0] == -math.inf
    else:
        check(o[1:], lse[1:], q[1:], [ks[1][:, 20:21]], [vs[1][:, 20:21]], 1.0 / math.sqrt(D), dtype, False)


def test_buffers_made_for_a_larger_batch():
    """Tables, lengths and outputs with more rows than q, or of another shape: the first B rows are used,
    as they always were."""
    D, H, dtype = 64, 2, torch.float16
    rng = np.random.default_rng(1)
    lens = [40, 7, 300, 16, 90]
    kc, vc, _, _, bt, sl, _, _ = fill(rng, lens, H, D, dtype, False)
    q = randn(len(lens), H, D, dtype=dtype)
    want, want_lse = fa.decode_paged(q[:3].contiguous(), kc, vc, bt[:3].contiguous(), sl[:3].contiguous())
    o, lse = fa.decode_paged(q[:3].contiguous(), kc, vc, bt, sl)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    out, out_lse = torch.full((5, H * D), 7.0, device="cuda", dtype=dtype), torch.full((5, H, 1), 7.0, device="cuda")
    o, lse = fa.decode_paged(q[:3].contiguous(), kc, vc, bt, sl[:, None], out=out, lse=out_lse)
    assert o is out and lse is out_lse and status() == fa.FA_OK
    assert torch.equal(out[:3].view(3, H, D), want) and torch.equal(out_lse[:3, :, 0], want_lse)
    assert torch.all(out[3:] == 7.0) and torch.all(out_lse[3:] == 7.0)
