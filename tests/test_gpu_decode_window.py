"""One decode step under a sliding window with first tokens that stay visible, against the definition in
64 bits over the visible rows (tolerances as derived in test_gpu_decode_gqa)."""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import PAGE, status
from test_gpu_decode_gqa import check, fill
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def visible(n, window, sinks):
    t = np.arange(n)
    return (t >= n - window) | (t < sinks)


def hide(lens, window, sinks, kc, vc, ke, ve, bt):
    """Table entries of pages without a visible token become bad ones, and hidden slots of the other
    pages NaN; returns the new table."""
    table = bt.cpu().numpy().copy()
    for b, n in enumerate(lens):
        see = visible(n, window, sinks)
        for pg in range((n + PAGE - 1) // PAGE):
            slots = np.zeros(PAGE, bool)
            part = see[pg * PAGE:(pg + 1) * PAGE]
            slots[:len(part)] = part
            page = table[b, pg]
            if not slots.any():
                table[b, pg] = -3
            elif not slots.all():
                gone = torch.from_numpy(~slots).cuda()
                for c, e in ((kc, ke), (vc, ve)):
                    if e is None:
                        c[page, :, gone] = math.nan
                    else:
                        c.view(torch.uint8)[page, :, gone] = 0x7f
                        e[page, :, gone] = 255
    return torch.from_numpy(table).cuda()


def run(seed, lens, Hq, Hk, D, dtype, q8, window, sinks, scale=None, extra=0):
    rng = np.random.default_rng(seed)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8)
    bt = hide(lens, window, sinks, kc, vc, ke, ve, bt)
    if extra:
        bt = torch.cat([bt, torch.full((bt.shape[0], extra), -7, dtype=torch.int32, device="cuda")], 1).contiguous()
    q = randn(len(lens), Hq, D, dtype=dtype)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, scale, k_exp=ke, v_exp=ve, window=window, sinks=sinks)
    assert status() == fa.FA_OK
    ks, vs = ([x[:, visible(n, window, sinks)] for x, n in zip(rows, lens)] for rows in (ks, vs))
    check(o, lse, q, ks, vs, scale if scale is not None else 1 / math.sqrt(D), dtype, q8)


BF16, FP16 = torch.bfloat16, torch.float16
LENS = [0, 1, 15, 16, 17, 33, 100, 257, 1000]


@pytest.mark.parametrize("extra", [0, 300], ids=["narrow", "wide"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 1), (100, 16), (31, 20), (64, 40), (5000, 3), (8, 2000)])
@pytest.mark.parametrize("Hq,Hk,D,dtype,q8", [(2, 2, 64, BF16, False), (8, 2, 128, FP16, False),
                                              (6, 2, 128, BF16, True), (16, 1, 64, FP16, True)])
def test_against_the_definition(Hq, Hk, D, dtype, q8, window, sinks, extra):
    run(1, LENS, Hq, Hk, D, dtype, q8, window, sinks, extra=extra)


@pytest.mark.parametrize("B,Hk,lens,window,sinks", [
    (300, 8, 700, 90, 5),     # three rounds of stretches
    (40, 2, 3000, 1500, 100),  # units that are cut
    (3, 1, 20000, 9000, 33),  # long ones
])
def test_many_and_long(B, Hk, lens, window, sinks):
    rng = np.random.default_rng(2)
    run(3, [int(x) for x in rng.integers(1, lens, B)], 2 * Hk, Hk, 64, BF16, True, window, sinks)


def test_one_window_for_all_is_the_plain_step():
    """Both within the tolerance (they may split the pages differently)."""
    rng = np.random.default_rng(4)
    lens = [5, 300, 77]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, 128, BF16, False)
    q = randn(3, 8, 128, dtype=BF16)
    for kw in ({}, dict(window=300), dict(window=1 << 40, sinks=1 << 40)):
        o, lse = fa.decode_paged(q, kc, vc, bt, sl, **kw)
        check(o, lse, q, ks, vs, 1 / math.sqrt(128), BF16, False)
    assert status() == fa.FA_OK


def test_equal_heads_and_a_negative_scale():
    run(5, [40, 333], 4, 4, 64, FP16, False, 50, 7, scale=-0.2)


def test_captured_and_replayed_as_sequences_grow():
    rng = np.random.default_rng(6)
    lens = [100, 30]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, 64, FP16, True)
    q = randn(2, 4, 64, dtype=FP16)
    sl.copy_(torch.tensor([60, 20]))
    ws = torch.empty(fa.fa_decode_window_workspace_bytes(2, 4, 2, 64, bt.shape[1], 24, 3), dtype=torch.uint8,
                     device="cuda")
    o, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    s = torch.cuda.Stream()

    def step():
        fa.decode_paged(q, kc, vc, bt, sl, out=o, lse=lse, workspace=ws, k_exp=ke, v_exp=ve, window=24, sinks=3)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for n in ([61, 21], lens):
        sl.copy_(torch.tensor(n))
        graph.replay()
        torch.cuda.synchronize()
        see = [[x[:, :m][:, visible(m, 24, 3)] for x, m in zip(rows, n)] for rows in (ks, vs)]
        check(o, lse, q, see[0], see[1], 1 / 8, FP16, True)
    assert status() == fa.FA_OK


def test_bad_lengths_and_pages_are_reported():
    rng = np.random.default_rng(7)
    kc, vc, ke, ve, bt, sl, _, _ = fill(rng, [100, 60], 1, 64, BF16, False)
    q = randn(2, 2, 64, dtype=BF16)
    for n, page in ((16 * bt.shape[1] + 1, None), (-1, None), (100, kc.shape[0]), (100, -1)):
        s2, b2 = sl.clone(), bt.clone()
        s2[0] = n
        if page is not None:
            b2[0, 6] = page  # the window's last page
        fa.decode_paged(q, kc, vc, b2, s2, window=20)
        assert status() == fa.FA_ERR_INVALID_ARG
    fa.decode_paged(q, kc, vc, bt, sl, window=20)
    assert status() == fa.FA_OK


def test_refusals():
    rng = np.random.default_rng(8)
    kc, vc, ke, ve, bt, sl, _, _ = fill(rng, [10], 1, 64, BF16, False)
    q = randn(1, 2, 64, dtype=BF16)
    for window, sinks in ((0, 0), (-4, 0), (4, -1)):
        with pytest.raises(fa.FaError):
            fa.decode_paged(q, kc, vc, bt, sl, window=window, sinks=sinks)
    with pytest.raises(fa.FaError):
        fa.decode_paged(q, kc, vc, bt, sl, window=4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        fa.decode_paged(q.half(), kc, vc, bt, sl, window=4)
