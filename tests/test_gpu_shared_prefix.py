"""A decode step over a shared prefix and own tokens against the definition in 64 bits.

Tolerance: that of test_gpu_decode_gqa.py.  In the prefix's kernel P lies between 2^-inf and 2^8 of
a running reference and is rounded to the 16-bit type like there; joining parts adds fp32
roundings alone (inside the 2^-20 of d).
"""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import PAGE, make_cache, status, tables
from test_gpu_decode_gqa import check
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def build(rng, prefix, lens, Hk, D, dtype):
    """A cache of NaN with the prefix's and the sequences' rows written; the rows in 64 bits."""
    t, pages = tables(rng, [prefix] + lens)
    kc, vc, _, _ = make_cache(pages, Hk, D, dtype, False)
    bt = torch.from_numpy(t).cuda()
    all_lens = [prefix] + lens
    ks, vs = [], []
    for b, n in enumerate(all_lens):
        k = torch.from_numpy(rng.standard_normal((1, Hk, max(n, 1), D), dtype=np.float32)).to(dtype).cuda()
        v = torch.from_numpy(rng.standard_normal((1, Hk, max(n, 1), D), dtype=np.float32)).to(dtype).cuda()
        n1 = torch.tensor([n], dtype=torch.int32, device="cuda")
        fa.cache_append(k, v, kc, vc, bt[b:b + 1].contiguous(), n1, n1)
        ks.append(gh.f64(k[0, :, :n]))
        vs.append(gh.f64(v[0, :, :n]))
    n_pre = (prefix + PAGE - 1) // PAGE
    own = max(1, (max(lens) + PAGE - 1) // PAGE)
    kk = [np.concatenate((ks[0], k), 1) for k in ks[1:]]
    vv = [np.concatenate((vs[0], v), 1) for v in vs[1:]]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return kc, vc, bt[0, :n_pre].contiguous(), bt[1:, :own].contiguous(), sl, kk, vv


CASES = [
    # prefix, own lengths, Hq, Hk, D, dtype
    (1, [0, 3], 2, 2, 64, torch.float16),
    (16, [1], 1, 1, 128, torch.bfloat16),
    (127, [5, 0, 17], 6, 2, 64, torch.bfloat16),       # group 3: 126 of 128 rows
    (128, [0, 0], 8, 1, 128, torch.float16),
    (129, [40, 1, 16, 100], 4, 4, 128, torch.bfloat16),
    (517, [0, 7, 45, 31], 16, 4, 64, torch.float16),
    (1000, [3] * 33, 8, 1, 128, torch.bfloat16),       # 264 rows: three query tiles, one pair half full
    (300, [2] * 130, 4, 4, 64, torch.bfloat16),        # 130 rows of group 1
    (2061, [9] * 20, 28, 2, 128, torch.float16),       # group 14, nine sequences a tile
    (400, [11, 70], 128, 1, 64, torch.bfloat16),       # one sequence a tile
    (700, [20, 5, 0], 17 * 3, 3, 128, torch.bfloat16),
    (0, [33, 0], 4, 2, 64, torch.bfloat16),            # no prefix
    (40, [1, 0, 19] * 400, 1, 1, 64, torch.float16),   # more sequences than one launch takes
    (150, [3000, 0, 40], 16, 1, 128, torch.float16),   # own tokens split over many warps
]


@pytest.mark.parametrize("prefix,lens,Hq,Hk,D,dtype", CASES, ids=lambda x: str(x).replace("torch.", "")[:20])
def test_shapes(prefix, lens, Hq, Hk, D, dtype):
    rng = np.random.default_rng(prefix + Hq)
    kc, vc, pt, bt, sl, ks, vs = build(rng, prefix, lens, Hk, D, dtype)
    q = randn(len(lens), Hq, D, dtype=dtype, seed=Hq)
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, prefix, bt, sl)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)


def test_no_tokens_of_their_own():
    """No page at all for the sequences (max_pages = 0), with and without a prefix."""
    D, dtype = 64, torch.float16
    rng = np.random.default_rng(1)
    kc, vc, pt, bt, sl, ks, vs = build(rng, 200, [0, 0, 0], 2, D, dtype)
    q = randn(3, 4, D, dtype=dtype)
    none = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, 200, none, sl)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, 0, none, sl)
    assert status() == fa.FA_OK
    assert not torch.any(o) and torch.isneginf(lse).all()


@pytest.mark.parametrize("scale", [1.0, -0.125, 0.0])
def test_scale(scale):
    D, dtype = 64, torch.bfloat16
    rng = np.random.default_rng(2)
    kc, vc, pt, bt, sl, ks, vs = build(rng, 333, [20, 0, 9], 2, D, dtype)
    q = randn(3, 8, D, dtype=dtype)
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, 333, bt, sl, scale)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, scale, dtype, False)


def test_prefix_shorter_than_its_table():
    """Tokens past prefix_len in the prefix's own pages, and pages past it, do not count."""
    D, dtype, Hk = 128, torch.bfloat16, 2
    rng = np.random.default_rng(3)
    kc, vc, pt, bt, sl, ks, vs = build(rng, 500, [12, 3], Hk, D, dtype)
    q = randn(2, 4, D, dtype=dtype)
    for n in (499, 385, 384, 130, 16, 1):
        o, lse = fa.decode_shared_prefix(q, kc, vc, pt, n, bt, sl)
        assert status() == fa.FA_OK
        cut = [np.concatenate((k[:, :n], k[:, 500:]), 1) for k in ks], [np.concatenate((v[:, :n], v[:, 500:]), 1) for v in vs]
        check(o, lse, q, *cut, 1.0 / math.sqrt(D), dtype, False)


def test_agrees_with_the_prefix_in_every_table():
    """The same step with the prefix's pages at the head of every sequence's own table (16 * k tokens)."""
    D, dtype, Hk, n = 128, torch.float16, 2, 48 * 16
    rng = np.random.default_rng(4)
    lens = [0, 100, 31, 5]
    kc, vc, pt, bt, sl, ks, vs = build(rng, n, lens, Hk, D, dtype)
    q = randn(4, 16, D, dtype=dtype)
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, n, bt, sl)
    whole = torch.cat((pt[None].expand(4, -1), bt), 1).contiguous()
    o2, lse2 = fa.decode_paged(q, kc, vc, whole, sl + n)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)
    check(o2, lse2, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)


def test_large_scores_and_rescaling():
    """Keys that grow along the prefix: the running reference is raised again and again, in the
    prefix's parts and between parts and own tokens."""
    D, dtype, Hk, prefix, lens = 64, torch.bfloat16, 1, 1500, [60, 10]
    rng = np.random.default_rng(5)
    t, pages = tables(rng, [prefix] + lens)
    kc, vc, _, _ = make_cache(pages, Hk, D, dtype, False)
    bt = torch.from_numpy(t).cuda()
    ks, vs = [], []
    for b, n in enumerate([prefix] + lens):
        k = torch.from_numpy(rng.standard_normal((1, Hk, n, D), dtype=np.float32))
        k = (k * torch.linspace(0.1, 6.0, n)[None, None, :, None]).to(dtype).cuda()
        v = randn(1, Hk, n, D, dtype=dtype, seed=b)
        n1 = torch.tensor([n], dtype=torch.int32, device="cuda")
        fa.cache_append(k, v, kc, vc, bt[b:b + 1].contiguous(), n1, n1)
        ks.append(gh.f64(k[0])), vs.append(gh.f64(v[0]))
    q = randn(2, 8, D, dtype=dtype) * 3
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.decode_shared_prefix(q, kc, vc, bt[0, :94].contiguous(), prefix, bt[1:, :4].contiguous(), sl)
    assert status() == fa.FA_OK
    check(o, lse, q, [np.concatenate((ks[0], k), 1) for k in ks[1:]],
          [np.concatenate((vs[0], v), 1) for v in vs[1:]], 1.0 / math.sqrt(D), dtype, False)


def test_repeated_captured_and_two_streams():
    """The same bits each time; two captured graphs with their own workspaces on two streams, with
    own lengths that changed after the capture."""
    D, dtype, Hk = 128, torch.bfloat16, 2
    rng = np.random.default_rng(6)
    kc, vc, pt, bt, sl, ks, vs = build(rng, 900, [50, 20, 64], Hk, D, dtype)
    q = randn(3, 8, D, dtype=dtype)
    first = fa.decode_shared_prefix(q, kc, vc, pt, 900, bt, sl)
    for _ in range(3):
        again = fa.decode_shared_prefix(q, kc, vc, pt, 900, bt, sl)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    need = fa.fa_shared_prefix_workspace_bytes(3, 8, Hk, D, 900, bt.shape[1])
    runs = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(q), torch.empty((3, 8), device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fa.decode_shared_prefix(q, kc, vc, pt, 900, bt, sl, out=o, lse=lse, workspace=ws)
        runs.append((graph, s, o, lse, ws))
    torch.cuda.synchronize()
    sl.copy_(torch.tensor([7, 20, 0], dtype=torch.int32))
    torch.cuda.synchronize()
    for graph, s, *_ in runs:
        with torch.cuda.stream(s):
            graph.replay()
    assert status() == fa.FA_OK
    cut = [x[:, :900 + n] for x, n in zip(ks, (7, 20, 0))], [x[:, :900 + n] for x, n in zip(vs, (7, 20, 0))]
    for _, _, o, lse, _ in runs:
        check(o, lse, q, *cut, 1.0 / math.sqrt(D), dtype, False)


def test_bad_device_data_is_reported():
    D, dtype = 64, torch.float16
    rng = np.random.default_rng(7)
    kc, vc, pt, bt, sl, ks, vs = build(rng, 150, [20, 3], 2, D, dtype)
    q = randn(2, 4, D, dtype=dtype)
    for at, page in ((0, kc.shape[0]), (9, -1)):
        bad = pt.clone()
        bad[at] = page
        fa.decode_shared_prefix(q, kc, vc, bad, 150, bt, sl)
        assert status() == fa.FA_ERR_INVALID_ARG
    bad = bt.clone()
    bad[0, 0] = 1 << 30
    fa.decode_shared_prefix(q, kc, vc, pt, 150, bad, sl)
    assert status() == fa.FA_ERR_INVALID_ARG
    fa.decode_shared_prefix(q, kc, vc, pt, 150, bt, sl + 1000)
    assert status() == fa.FA_ERR_INVALID_ARG
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, 150, bt, sl)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)


def test_refusals_of_the_public_call():
    D = 64
    q = randn(2, 4, D, dtype=torch.float16)
    kc, vc, ke, ve = make_cache(4, 2, D, torch.float16, False)
    bt = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    sl = torch.zeros(2, dtype=torch.int32, device="cuda")
    pt = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fa.decode_shared_prefix(q, kc, vc, pt, 33, bt, sl)       # the table holds 32 tokens
    with pytest.raises(ValueError):
        fa.decode_shared_prefix(q, kc, vc, pt, -1, bt, sl)
    with pytest.raises(TypeError):
        fa.decode_shared_prefix(q, kc, vc, pt.long(), 16, bt, sl)
    with pytest.raises(TypeError):
        fa.decode_shared_prefix(q.bfloat16(), kc, vc, pt, 16, bt, sl)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(fa.FaError):
        fa.decode_shared_prefix(q, kc, vc, pt, 16, bt, sl, workspace=small)
    assert status() == fa.FA_OK
