"""Attention of chunks of new tokens over a paged cache against the definition in 64 bits over the rows as
the cache holds them, with tolerances derived in window_reference."""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import PAGE, make_cache, status
from test_gpu_decode_gqa import fill
from test_gpu_rotary import randn
from window_reference import reference, sees, within

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def hide(lens, news, window, sinks, kc, vc, ke, ve, bt):
    """Table entries of pages without a token that some row sees become bad ones, and slots of the other
    pages that hold none NaN."""
    table = bt.cpu().numpy().copy()
    for b, (n, new) in enumerate(zip(lens, news)):
        t = np.arange(n)
        live = (t < sinks) | (t > n - new - window) if window else np.ones(n, bool)
        live &= new > 0
        for pg in range((n + PAGE - 1) // PAGE):
            slots = np.zeros(PAGE, bool)
            part = live[pg * PAGE:(pg + 1) * PAGE]
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


def check(o, lse, q, ks, vs, lens, news, window, sinks, scale):
    Hq, L = q.shape[1:3]
    for b, (n, new) in enumerate(zip(lens, news)):
        assert not o[b, :, new:].any() and (lse[b, :, new:] == -math.inf).all(), b
        if new == 0:
            continue
        Hk = ks[b].shape[0]
        G = Hq // Hk
        mask = sees(new, n, window or n, sinks if window else 0)
        for h in range(Hk):
            heads = slice(h * G, h * G + G)
            k, v = (torch.from_numpy(np.ascontiguousarray(x[b][h])).cuda() for x in (ks, vs))
            want = reference(q[b, heads, :new], k, v, mask, scale)
            within(o[b, heads, :new], want["o"], f"o[{b}, {h}]")
            within(lse[b, heads, :new], want["lse"], f"lse[{b}, {h}]")


def run(seed, lens, news, Hq, Hk, D, dtype, q8, window=0, sinks=0, scale=None, L=None, layout="bhld", scale_rows=None):
    rng = np.random.default_rng(seed)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8, scale_rows)
    bt = hide(lens, news, window, sinks, kc, vc, ke, ve, bt)
    B, L = len(lens), L or max(max(news), 1)
    q = randn(B, Hq, L, D, dtype=dtype, seed=seed)
    if layout == "blhd":
        q = q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.full_like(q, math.nan)
    nl = torch.tensor(news, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks) if window else {}
    o, lse = fa.attention_paged(q, kc, vc, bt, sl, nl, scale=scale, out=out, k_exp=ke, v_exp=ve, **kw)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, lens, news, window, sinks, scale if scale is not None else 1 / math.sqrt(D))


LENS = [0, 1, 17, 16, 300, 1000, 129, 640]
NEWS = [0, 1, 17, 0, 5, 130, 128, 100]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (64, 3), (200, 40), (130, 150)])
@pytest.mark.parametrize("Hq,Hk,D,dtype,q8", [
    (2, 2, 64, BF16, False), (8, 2, 128, FP16, False), (6, 2, 128, BF16, False), (16, 1, 64, FP16, False),
    (3, 3, 128, BF16, True), (8, 2, 64, FP16, True), (5, 1, 64, BF16, True), (16, 2, 128, FP16, True)])
def test_against_the_definition(Hq, Hk, D, dtype, q8, window, sinks):
    run(1, LENS, NEWS, Hq, Hk, D, dtype, q8, window, sinks)


@pytest.mark.parametrize("lens,news,Hq,Hk,window,sinks,q8", [
    ([9000], [16], 4, 1, 0, 0, True),             # a few rows on a long cache: every CTA a stretch of it
    ([9000], [16], 4, 1, 0, 0, False),
    ([20000, 40], [257, 3], 8, 2, 0, 0, False),
    ([5000, 3000, 77], [1500, 2000, 77], 8, 4, 700, 5, True),
    ([2500], [2500], 2, 2, 0, 0, False),          # a prompt from its start
    ([2500], [2500], 2, 2, 300, 129, False),
    ([1], [1], 1, 1, 0, 0, False),
    ([4096] * 3, [1] * 3, 8, 8, 0, 0, True),      # single tokens
])
def test_splits(lens, news, Hq, Hk, window, sinks, q8):
    run(2, lens, news, Hq, Hk, 128, BF16, q8, window, sinks)


# Few rows per cache head are queries of the decode kernel: a cluster per unit or the line, one or two blocks of
# eight, two units of them over e4m3, and on either side of its limits of 16 and 32 rows.
FEW = [(1, 1, 1), (3, 3, 5), (8, 2, 2), (8, 2, 4), (6, 2, 5), (5, 1, 3), (2, 2, 16), (2, 2, 17), (16, 2, 4), (11, 1, 3)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 40), (64, 3), (200, 0)])
@pytest.mark.parametrize("D,dtype,q8", [(64, BF16, False), (128, FP16, False), (128, BF16, True), (64, FP16, True)])
@pytest.mark.parametrize("Hq,Hk,L", FEW)
def test_few_rows(Hq, Hk, L, D, dtype, q8, window, sinks):
    lens = [0, 1, 17, 16, 300, 1000, 129, 640, L, 64 + L]
    news = [0, 1, min(L, 17), 0, L, (L + 1) // 2, L, 1, L, L]
    run(21, lens, news, Hq, Hk, D, dtype, q8, window, sinks, L=L)


@pytest.mark.parametrize("lens,new,Hq,Hk,window,sinks,layout", [
    ([9000], 4, 8, 2, 0, 0, "blhd"),              # every warp a stretch of one sequence
    ([3000, 20, 4], 4, 4, 4, 0, 0, "blhd"),
    ([700] * 40, 3, 8, 4, 500, 20, "blhd"),       # clusters of several sizes
    ([700] * 200, 2, 4, 2, 100, 0, "bhld"),
    ([4000, 50] * 60, 5, 12, 4, 0, 0, "blhd"),    # the line
    ([40] * 1100, 2, 2, 1, 0, 0, "blhd"),         # two launches
])
@pytest.mark.parametrize("q8", [False, True])
def test_few_rows_splits(lens, new, Hq, Hk, window, sinks, layout, q8):
    run(22, lens, [new] * len(lens), Hq, Hk, 128, BF16, q8, window, sinks, layout=layout)


@pytest.mark.parametrize("q8", [False, True])
def test_few_rows_whose_padding_holds_nan(q8):
    rng = np.random.default_rng(23)
    lens, news = [300, 20, 5000], [3, 0, 1]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, 128, BF16, q8)
    q = randn(3, 4, 4, 128, dtype=BF16)
    for b, n in enumerate(news):
        q[b, :, n:] = math.nan
    nl = torch.tensor(news, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_paged(q, kc, vc, bt, sl, nl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, lens, news, 0, 0, 1 / math.sqrt(128))


def test_one_new_token_is_a_decode_step():
    rng = np.random.default_rng(24)
    kc, vc, ke, ve, bt, sl, _, _ = fill(rng, [300, 1, 5000, 77], 2, 128, BF16, True)
    q = randn(4, 8, 1, 128, dtype=BF16)
    kw = dict(window=200, sinks=9, k_exp=ke, v_exp=ve)
    o, lse = fa.attention_paged(q, kc, vc, bt, sl, **kw)
    od, lsed = fa.decode_paged(q[:, :, 0].contiguous(), kc, vc, bt, sl, **kw)
    assert torch.equal(o[:, :, 0], od) and torch.equal(lse[:, :, 0], lsed)


@pytest.mark.parametrize("q8", [False, True])
def test_few_rows_with_bad_lengths(q8):
    rng = np.random.default_rng(25)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, [100, 60], 1, 64, BF16, q8)
    q = randn(2, 2, 4, 64, dtype=BF16)
    kw = dict(k_exp=ke, v_exp=ve)
    for n, new in ((16 * bt.shape[1] + 1, 4), (-1, 0), (3, 4), (100, 5), (100, -1)):
        s2 = torch.tensor([n, 60], dtype=torch.int32, device="cuda")
        nl = torch.tensor([new, 4], dtype=torch.int32, device="cuda")
        o, lse = fa.attention_paged(q, kc, vc, bt, s2, nl, **kw)
        assert status() == fa.FA_ERR_INVALID_ARG, (n, new)
        check(o[1:], lse[1:], q[1:], ks[1:], vs[1:], [60], [4], 0, 0, 1 / 8)
        assert not o[0].any() and (lse[0] == -math.inf).all()
    for page in (kc.shape[0], -1):
        b2 = bt.clone()
        b2[0, 3] = page
        o, lse = fa.attention_paged(q, kc, vc, b2, sl, **kw)
        assert status() == fa.FA_ERR_INVALID_ARG, page
        check(o[1:], lse[1:], q[1:], ks[1:], vs[1:], [60], [4], 0, 0, 1 / 8)


@pytest.mark.parametrize("pages", [64, 2000])
def test_few_rows_captured_and_replayed_on_a_side_stream(pages):
    """Lengths and counts change between replays; a cluster per unit (a short table) and the line."""
    rng = np.random.default_rng(26)
    lens, news = [900, 130, 3], [4, 1, 3]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, 64, FP16, True)
    bt = torch.nn.functional.pad(bt, (0, pages - bt.shape[1])).contiguous()
    q = randn(3, 4, 4, 64, dtype=FP16)
    nl, o, lse = torch.ones(3, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty(3, 4, 4, device="cuda")
    ws = torch.empty(fa.fa_attention_paged_workspace_bytes(3, 4, 2, 4, 64, pages), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()

    def step():
        fa.attention_paged(q, kc, vc, bt, sl, nl, out=o, lse=lse, workspace=ws, k_exp=ke, v_exp=ve)

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for n, m in (([400, 0, 1], [4, 0, 1]), (lens, news)):
        sl.copy_(torch.tensor(n))
        nl.copy_(torch.tensor(m))
        graph.replay()
        torch.cuda.synchronize()
        check(o, lse, q, [x[:, :a] for x, a in zip(ks, n)], [x[:, :a] for x, a in zip(vs, n)], n, m, 0, 0, 1 / 8)
    assert status() == fa.FA_OK


@pytest.mark.parametrize("Hq,Hk", [(128, 1), (100, 1), (65, 1), (64, 2)])
def test_large_groups(Hq, Hk):
    run(3, [70, 300], [20, 9], Hq, Hk, 64, FP16, False)


def test_many_sequences():
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 200, 700)]
    news = [int(rng.integers(0, min(n, 8) + 1)) for n in lens]
    run(5, lens, news, 2, 1, 64, BF16, True)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
@pytest.mark.parametrize("q8", [False, True])
def test_scales_and_layout(scale, q8):
    run(6, [200, 333], [70, 100], 4, 2, 64, FP16, q8, 0, 0, scale, L=111, layout="blhd")


def test_rows_of_very_different_size():
    """e4m3 rows whose powers of two lie far apart (the values stay in fp16's range)."""
    def scales(rng, shape):
        return np.exp2(rng.integers(-10, 10, shape)).astype(np.float32)
    run(7, [300], [40], 4, 2, 64, FP16, True, scale_rows=scales)
    run(7, [300], [40], 4, 2, 128, BF16, True, scale_rows=scales)


def test_all_rows_new_without_new_lens():
    rng = np.random.default_rng(8)
    lens = [40, 0, 90]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, 64, BF16, False)
    q = randn(3, 4, 33, 64, dtype=BF16)
    o, lse = fa.attention_paged(q, kc, vc, bt, sl)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, lens, [33, 0, 33], 0, 0, 1 / 8)


def test_the_same_bits_every_time():
    rng = np.random.default_rng(9)
    kc, vc, ke, ve, bt, sl, _, _ = fill(rng, [5000, 700], 2, 128, BF16, True)
    q = randn(2, 8, 300, 128, dtype=BF16)
    a = fa.attention_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    for _ in range(3):
        b = fa.attention_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q8", [False, True])
def test_offsets_past_31_bits(q8):
    """Pages at the far end of a cache of more than 2^31 elements."""
    Hk, D, n, new = 8, 128, 100, 40
    pages = (1 << 31) // (Hk * PAGE * D) + 16
    kc, vc = (torch.empty((pages, Hk, PAGE, D), device="cuda", dtype=torch.float8_e4m3fn if q8 else BF16) for _ in range(2))
    ke, ve = ((torch.zeros((pages, Hk, PAGE), device="cuda", dtype=torch.uint8) for _ in range(2)) if q8 else (None, None))
    bt = torch.arange(pages - 7, pages, dtype=torch.int32, device="cuda")[None].contiguous()
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    k, v = randn(1, Hk, n, D, dtype=BF16, seed=1), randn(1, Hk, n, D, dtype=BF16, seed=2)
    fa.cache_append(k, v, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    kd, vd = fa.cache_read(kc, vc, bt, sl, n, k_exp=ke, v_exp=ve, dtype=BF16)
    q = randn(1, 16, new, D, dtype=BF16, seed=3)
    o, lse = fa.attention_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    od, lsed = fa.decode_paged(q[:, :, -1].contiguous(), kc, vc, bt, sl, k_exp=ke, v_exp=ve, window=60, sinks=4)
    assert status() == fa.FA_OK
    check(o, lse, q, [gh.f64(kd[0])], [gh.f64(vd[0])], [n], [new], 0, 0, 1 / math.sqrt(D))
    mask = sees(1, n, 60, 4)
    for h in range(Hk):
        want = reference(q[0, 2 * h:2 * h + 2, -1:], kd[0, h], vd[0, h], mask, 1 / math.sqrt(D))
        within(od[0, 2 * h:2 * h + 2, None], want["o"], "decode o")


def test_rows_past_31_bits_without_a_token():
    """More than 2^28 rows of which a few are new (q's rows overlap in memory, O's do not)."""
    D, n, new, L = 64, 100, 40, (1 << 28) + 100
    kc, vc = (randn(8, 1, PAGE, D, dtype=BF16, seed=s) for s in (1, 2))
    bt = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    sl, nl = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (n, new))
    rows = randn(8 * L + D, dtype=BF16, seed=3)
    q = rows.as_strided((1, 1, L, D), (8 * L, 8 * L, 8, 1))
    o = torch.empty((1, 1, L, D), device="cuda", dtype=BF16)
    o[:, :, :256] = o[:, :, -256:] = math.nan
    lse = fa.attention_paged(q, kc, vc, bt, sl, nl, out=o)[1]
    assert status() == fa.FA_OK
    k, v = (x.reshape(1, 8 * PAGE, D)[:, :n] for x in (kc, vc))
    check(o[:, :, :256], lse[:, :, :256], q[:, :, :256], [gh.f64(k)], [gh.f64(v)], [n], [new], 0, 0, 1 / math.sqrt(D))
    assert not o[:, :, -256:].any() and (lse[:, :, new:] == -math.inf).all()
    del o, lse, rows, q
    torch.cuda.empty_cache()


def test_captured_and_replayed_as_sequences_grow():
    rng = np.random.default_rng(10)
    lens, news = [900, 130], [64, 30]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, 64, FP16, True)
    q = randn(2, 8, 64, 64, dtype=FP16)
    nl = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    sl.copy_(torch.tensor([64, 64]))
    ws = torch.empty(fa.fa_attention_paged_workspace_bytes(2, 8, 2, 64, 64, bt.shape[1]), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(2, 8, 64, device="cuda")
    s = torch.cuda.Stream()

    def step():
        fa.attention_paged(q, kc, vc, bt, sl, nl, out=o, lse=lse, workspace=ws, k_exp=ke, v_exp=ve)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for n, m in (([400, 0], [64, 0]), (lens, news)):
        sl.copy_(torch.tensor(n))
        nl.copy_(torch.tensor(m))
        graph.replay()
        torch.cuda.synchronize()
        check(o, lse, q, [x[:, :a] for x, a in zip(ks, n)], [x[:, :a] for x, a in zip(vs, n)], n, m, 0, 0, 1 / 8)
    assert status() == fa.FA_OK


@pytest.mark.parametrize("q8", [False, True])
def test_bad_lengths_and_pages_are_reported(q8):
    rng = np.random.default_rng(11)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, [100, 60], 1, 64, BF16, q8)
    q = randn(2, 2, 20, 64, dtype=BF16)
    kw = dict(k_exp=ke, v_exp=ve)
    for n, new in ((16 * bt.shape[1] + 1, 20), (-1, 0), (10, 20), (100, 21), (100, -1)):
        s2 = torch.tensor([n, 60], dtype=torch.int32, device="cuda")
        nl = torch.tensor([new, 20], dtype=torch.int32, device="cuda")
        o, lse = fa.attention_paged(q, kc, vc, bt, s2, nl, **kw)
        assert status() == fa.FA_ERR_INVALID_ARG, (n, new)
        check(o[1:], lse[1:], q[1:], ks[1:], vs[1:], [60], [20], 0, 0, 1 / 8)  # the other one is right
        assert not o[0].any()
    for page in (kc.shape[0], -1, 1 << 30):
        b2 = bt.clone()
        b2[0, 3] = page
        o, lse = fa.attention_paged(q, kc, vc, b2, sl, **kw)
        assert status() == fa.FA_ERR_INVALID_ARG, page
        check(o[1:], lse[1:], q[1:], ks[1:], vs[1:], [60], [20], 0, 0, 1 / 8)
    fa.attention_paged(q, kc, vc, bt, sl, **kw)
    assert status() == fa.FA_OK


def test_no_sequence_has_tokens():
    kc, vc, ke, ve = make_cache(2, 1, 64, BF16, False)
    bt = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    sl = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = randn(3, 2, 5, 64, dtype=BF16)
    for table in (bt, torch.full((3, 4), -1, dtype=torch.int32, device="cuda")):
        o, lse = fa.attention_paged(q, kc, vc, table, sl)
        assert not o.any() and (lse == -math.inf).all()
    assert status() == fa.FA_OK


def test_refusals():
    rng = np.random.default_rng(12)
    kc, vc, ke, ve, bt, sl, _, _ = fill(rng, [40], 2, 64, BF16, False)
    q = randn(1, 4, 8, 64, dtype=BF16)
    with pytest.raises(ValueError):
        fa.attention_paged(q, kc, vc, bt, sl, window=0)
    with pytest.raises(fa.FaError):
        fa.attention_paged(q, kc, vc, bt, sl, window=4, sinks=-1)
    with pytest.raises(fa.FaError):
        fa.attention_paged(q[:, :3], kc, vc, bt, sl)
    with pytest.raises(fa.FaError):
        fa.attention_paged(q, kc, vc, bt, sl, out=q)
    with pytest.raises(fa.FaError):
        fa.attention_paged(q, kc, vc, bt, sl, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        fa.attention_paged(q.half(), kc, vc, bt, sl)
    with pytest.raises(ValueError):
        fa.attention_paged(q, kc, vc, bt, sl, torch.tensor([8], device="cuda"))
    with pytest.raises(ValueError):
        fa.attention_paged(q[0], kc, vc, bt, sl)
    with pytest.raises(ValueError):
        fa.attention_paged(q, kc, vc, bt, sl, lse=torch.empty(1, 4, 7, device="cuda"))
    many = randn(1, 258, 2, 64, dtype=BF16)
    with pytest.raises(fa.FaError):  # groups of more than 128 heads
        fa.attention_paged(many, kc, vc, bt, sl)
    assert status() == fa.FA_OK


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_prompt_in_chunks_then_tokens(window, sinks):
    """A prompt is written and attended to in chunks, then single tokens follow: every row as one dense call
    over the whole sequence gives it (both within the tolerance of the definition)."""
    B, Hq, Hk, D, dtype, total = 2, 8, 2, 128, BF16, 300
    q, k, v = (randn(B, H, total, D, dtype=dtype, seed=s) for s, H in enumerate((Hq, Hk, Hk)))
    freqs, mscale = fa.rotary_freqs(D)
    q, kr = fa.rotary(q, k, None, freqs, mscale)
    lens = [total, total - 37]
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    bt = torch.zeros((B, max(pages)), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(pages)).to(torch.int32).cuda()
    bt[0, :pages[0]], bt[1, :pages[1]] = order[:pages[0]], order[pages[0]:]
    kc, vc, _, _ = make_cache(sum(pages), Hk, D, dtype, False)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, total, device="cuda")
    done = [0, 0]
    kw = dict(window=window, sinks=sinks) if window else {}
    for chunk in (128, 100, 40, 1, 1, 30):
        news = [min(chunk, n - d) for n, d in zip(lens, done)]
        nl = torch.tensor(news, dtype=torch.int32, device="cuda")
        sl = torch.tensor([d + n for d, n in zip(done, news)], dtype=torch.int32, device="cuda")
        part = [torch.zeros(B, H, chunk, D, device="cuda", dtype=dtype) for H in (Hq, Hk, Hk)]
        for b in range(B):
            for x, full in zip(part, (q, k, v)):
                x[b, :, :news[b]] = full[b, :, done[b]:done[b] + news[b]]
        fa.cache_append(part[1], part[2], kc, vc, bt, sl, nl, freqs=freqs, mscale=mscale)
        if chunk == 1 and min(news) == 1:
            oc, lc = fa.decode_paged(part[0][:, :, 0].contiguous(), kc, vc, bt, sl, **kw)
            oc, lc = oc[:, :, None], lc[:, :, None]
        else:
            oc, lc = fa.attention_paged(part[0], kc, vc, bt, sl, nl, **kw)
        for b in range(B):
            o[b, :, done[b]:done[b] + news[b]] = oc[b, :, :news[b]]
            lse[b, :, done[b]:done[b] + news[b]] = lc[b, :, :news[b]]
            done[b] += news[b]
    assert status() == fa.FA_OK and done == lens
    dense, dense_lse = fa.window_forward(q, kr, v, window or total, sinks)
    mask = sees(total, total, window or total, sinks)
    for b in range(B):
        n = lens[b]
        for h in range(Hk):
            heads = slice(4 * h, 4 * h + 4)
            want = reference(q[b, heads, :n], kr[b, h, :n], v[b, h, :n], mask[:n, :n], 1 / math.sqrt(D))
            for got, name in ((o, "o"), (lse, "lse"), (dense, "o"), (dense_lse, "lse")):
                within(got[b, heads, :n], want[name], f"{name}[{b}, {h}]")
