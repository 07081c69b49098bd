"""One decode step with grouped heads over a 16-bit or e4m3 cache against the definition in 64 bits.

Tolerance, element by element.  With weights p_j (softmax) and A = sum_j p_j |v_j|:
* a score is a sum of D exact products in fp32, off by at most D 2^-23 sum_i |q_i k_i| |scale|;
  d = the largest such error over the row's keys, plus 2^-20 for the exponentials (2^-22 each) and
  the sums, changes a weight by a factor within 1 + 2d (for small d) and its share by twice that;
* P is rounded to 16 bits, half a step: eps_P/2 of each weight (eps_P of fp16 for an e4m3 cache), or,
  below fp16's normal range, 2^-25 of the row's reference, which is at most its largest weight
  (times the row's scale for e4m3): n keys lose at most n 2^-25 of the largest term;
* O is rounded once: eps/2 |O| (and 2^-25 in fp16).
LSE is off by at most d, and its own fp32 rounding.
"""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import PAGE, held, make_cache, quantise, status, tables
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


EXTRA = 0


@pytest.fixture(scope="module", autouse=True, params=[0, 300], ids=["narrow", "wide"])
def _extra(request):
    """Everything with tables as long as they need to be (short steps take a cluster per head), and
    with 300 more columns, which no kernel may read (all steps take the split over all warps)."""
    global EXTRA
    EXTRA = request.param
    yield


def widen(bt, extra=None):
    n = EXTRA if extra is None else extra
    return torch.cat([bt, torch.full((bt.shape[0], n), -7, dtype=torch.int32, device="cuda")], 1).contiguous()


def fill(rng, lens, Hk, D, dtype, q8, scale_rows=None):
    """A cache whose pages hold the sequences' rows and NaN everywhere else, and the rows as held:
    lists of [Hk, n, D] in 64 bits."""
    t, pages = tables(rng, lens)
    kc, vc, ke, ve = make_cache(pages, Hk, D, dtype, q8)
    bt = widen(torch.from_numpy(t).cuda())
    L = max(max(lens), 1)
    k = torch.from_numpy(rng.standard_normal((len(lens), Hk, L, D), dtype=np.float32))
    v = torch.from_numpy(rng.standard_normal((len(lens), Hk, L, D), dtype=np.float32))
    if scale_rows is not None:
        v = v * torch.from_numpy(scale_rows(rng, tuple(v.shape[:3])))[..., None]
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fa.cache_append(k, v, kc, vc, bt, sl, sl, k_exp=ke, v_exp=ve)
    rows = []
    for x, c, e in ((k, kc, ke), (v, vc, ve)):
        rows.append([(quantise(gh.f64(x[b, :, :n]))[0] if q8 else gh.f64(x[b, :, :n])) if n else
                     np.zeros((Hk, 0, D)) for b, n in enumerate(lens)])
    return kc, vc, ke, ve, bt, sl, rows[0], rows[1]


def check(o, lse, q, ks, vs, scale, dtype, q8, mixed=False):
    """o [B, Hq, D], lse [B, Hq] against rows ks[b], vs[b] [Hk, n, D]."""
    eps = torch.finfo(dtype).eps
    epsp = torch.finfo(torch.float16).eps if q8 else eps
    if mixed:
        epsp = eps
    o, lse, q = gh.f64(o), gh.f64(lse), gh.f64(q)
    for b in range(q.shape[0]):
        Hk, n, D = ks[b].shape
        G = q.shape[1] // Hk
        for h in range(q.shape[1]):
            k, v = ks[b][h // G], vs[b][h // G]
            if n == 0:
                assert not np.any(o[b, h]) and np.isneginf(lse[b, h]), (b, h)
                continue
            s = scale * (k @ q[b, h])
            top = s.max()
            p = np.exp(s - top)
            l = p.sum()
            p /= l
            d = D * 2.0 ** -23 * abs(scale) * float((np.abs(k) @ np.abs(q[b, h])).max()) + 2.0 ** -20
            ref_lse = top + math.log(l)
            assert abs(lse[b, h] - ref_lse) <= d + abs(ref_lse) * 2.0 ** -22, (b, h, lse[b, h], ref_lse)
            ref = p @ v
            amax = np.abs(v).max(1)
            lost = n * 2.0 ** -24 * (float((p * amax).max()) if q8 else float(p.max() * amax.max()))
            bound = (epsp / 2 + 4 * d) * (p @ np.abs(v)) + lost + eps / 2 * np.abs(ref) * (1 + epsp) + 2.0 ** -25
            err = np.abs(o[b, h] - ref)
            assert np.all(err <= bound), (b, h, n, float((err / bound).max()))


@pytest.mark.parametrize("q8", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16), (64, torch.bfloat16),
                                     (128, torch.float16)], ids=str)
@pytest.mark.parametrize("Hq,Hk", [(3, 3), (8, 2), (8, 1), (10, 1), (36, 3), (40, 2)])
def test_shapes(q8, D, dtype, Hq, Hk):
    rng = np.random.default_rng(Hq * 100 + D)
    lens = [0, 1, 15, 16, 17, 63, 64, 129, 300, 1000]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8)
    q = randn(len(lens), Hq, D, dtype=dtype, seed=Hq)
    scale = 1.0 / math.sqrt(D)
    if Hq == Hk and not q8:  # equal heads on a 16-bit cache: the C entry itself
        o, lse = fa._decode_paged_ex(q, kc, vc, bt, sl, scale, None, None, None, None, None)
    else:
        o, lse = fa.decode_paged(q, kc, vc, bt, sl, scale, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, scale, dtype, q8)


@pytest.mark.parametrize("lens,Hq,Hk,q8", [([5000], 8, 1, True), ([70000], 4, 1, True),
                                           ([20000, 3], 12, 1, False), ([2000, 0], 4, 4, True),
                                           ([17, 4096, 1], 16, 1, False), ([1], 2, 2, True),
                                           ([0], 2, 1, True)])
def test_split_and_merge(lens, Hq, Hk, q8):
    D, dtype = 128, torch.bfloat16
    rng = np.random.default_rng(len(lens))
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8)
    q = randn(len(lens), Hq, D, dtype=dtype)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, q8)
    wide = torch.zeros((len(lens), 4 * bt.shape[1] + 40), dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt  # a table much wider than the sequences: more warps than pages
    o2, lse2 = fa.decode_paged(q, kc, vc, wide, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o2, lse2, q, ks, vs, 1.0 / math.sqrt(D), dtype, q8)


@pytest.mark.parametrize("scale", [1.0, -0.125, 0.0, 3.0])
@pytest.mark.parametrize("q8", [True, False], ids=["e4m3", "16bit"])
def test_scale(scale, q8):
    D, dtype, lens = 64, torch.float16, [40, 333]
    rng = np.random.default_rng(5)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, D, dtype, q8)
    q = randn(2, 8, D, dtype=dtype)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, scale, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, scale, dtype, q8)


def test_value_rows_of_very_different_magnitudes():
    """Value rows from 2^-60 to 2^60: a row's weight and its scale are taken together."""
    D, dtype, lens = 128, torch.bfloat16, [50, 400]
    rng = np.random.default_rng(6)

    def spread(r, shape):
        return np.ldexp(1.0, r.integers(-60, 61, shape)).astype(np.float32)

    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, D, dtype, True, spread)
    q = randn(2, 4, D, dtype=dtype) * 4
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, True)
    tiny = lambda r, shape: np.full(shape, 2.0 ** -100, dtype=np.float32)  # noqa: E731
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 2, D, dtype, True, tiny)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    ref = np.exp(1.0 / math.sqrt(D) * (ks[1][0] @ gh.f64(q[1, 0])))
    ref = (ref / ref.sum()) @ vs[1][0]
    assert status() == fa.FA_OK
    assert np.all(np.abs(gh.f64(o[1, 0]) - ref) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -110)


@pytest.mark.parametrize("power", [-90, -20, 30, 100])
def test_query_rows_of_any_magnitude(power):
    """bf16 queries far outside fp16's range over an e4m3 cache (the scale brings the scores back)."""
    D, dtype, lens = 64, torch.bfloat16, [70]
    rng = np.random.default_rng(7)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 1, D, dtype, True)
    q = (randn(1, 8, D, dtype=torch.float32).double() * 2.0 ** power).to(dtype)
    q[0, 3] = 0
    scale = 0.125 * 2.0 ** -power if abs(power) < 100 else 0.125 * 2.0 ** -power
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, scale, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, scale, dtype, True)


@pytest.mark.parametrize("q8", [True, False], ids=["e4m3", "16bit"])
def test_scores_of_any_size(q8):
    """Scores around -1e33 and 1e33 (far outside the exponentials' range) and rows of one huge key."""
    D, dtype, Hk = 64, torch.bfloat16, 1
    kc, vc, ke, ve = make_cache(2, Hk, D, dtype, q8)
    k = torch.zeros((2, Hk, 16, D), device="cuda", dtype=dtype)
    k[:, :, :, 0] = 2.0 ** 40
    k[:, :, 5, 0] = 2.0 ** 40 * 1.25   # the one key that counts (sign of q decides)
    v = randn(2, Hk, 16, D, dtype=dtype)
    bt = widen(torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"))
    sl = torch.tensor([16, 1], dtype=torch.int32, device="cuda")
    fa.cache_append(k, v, kc, vc, bt, torch.full_like(sl, 16), k_exp=ke, v_exp=ve)
    held_v = gh.f64(fa.cache_read(kc, vc, bt, torch.full_like(sl, 16), 16, k_exp=ke, v_exp=ve, dtype=dtype)[1])
    q = torch.zeros((2, 2, D), device="cuda", dtype=dtype)
    q[:, 0, 0], q[:, 1, 0] = 2.0 ** 70, -(2.0 ** 70)
    o, lse = fa._decode_paged_ex(q, kc, vc, bt, sl, 1.0, None, None, None, ke, ve)
    assert status() == fa.FA_OK
    big = 2.0 ** 110
    o, lse = gh.f64(o), gh.f64(lse)
    assert np.array_equal(o[0, 0], held_v[0, 0, 5]) and abs(lse[0, 0] / big - 1.25) <= 2.0 ** -22
    # the others tie: the mean of 15 rows (P is exact: 1 and 0)
    mean = held_v[0, 0][[i for i in range(16) if i != 5]].mean(0)
    assert np.all(np.abs(o[0, 1] - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -18)
    assert abs(lse[0, 1] / big + 1.0) <= 2.0 ** -22
    for h, s in ((0, 1.0), (1, -1.0)):  # one key alone, whatever its score
        assert np.array_equal(o[1, h], held_v[1, 0, 0]) and abs(lse[1, h] / big - s) <= 2.0 ** -22


def test_a_bad_row_stays_with_its_sequence_and_head():
    """A NaN key, an infinite value: the results of that sequence's head, no others'."""
    D, dtype, lens, Hk = 64, torch.bfloat16, [40, 40, 40], 2
    rng = np.random.default_rng(8)
    for q8 in (True, False):
        kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8)
        q = randn(3, 4, D, dtype=dtype)
        good, good_lse = fa._decode_paged_ex(q, kc, vc, bt, sl, None, None, None, None, ke, ve)
        page = int(bt[1, 1])
        if q8:
            ke[page, 1, 3] = 255
        else:
            kc[page, 1, 3, 5] = math.nan
        o, lse = fa._decode_paged_ex(q, kc, vc, bt, sl, None, None, None, None, ke, ve)
        assert torch.isnan(o[1, 2:]).all() and torch.isnan(lse[1, 2:]).all()
        keep = torch.ones(3, 4, dtype=torch.bool)
        keep[1, 2:] = False
        assert torch.equal(o[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])
        page = int(bt[0, 0])
        if q8:
            ve[page, 0, 0] = 255
        else:
            vc[page, 0, 0, 7] = math.inf
        o, lse = fa._decode_paged_ex(q, kc, vc, bt, sl, None, None, None, None, ke, ve)
        assert status() == fa.FA_OK
        assert not torch.isfinite(o[0, :2, 7]).any() and torch.equal(lse[0], good_lse[0])
        assert torch.equal(o[0, 2:], good[0, 2:]) and torch.equal(o[2], good[2])


def test_bad_device_data_is_reported():
    D, dtype, Hk = 128, torch.bfloat16, 2
    rng = np.random.default_rng(9)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, [40, 20], Hk, D, dtype, True)
    q = randn(2, 4, D, dtype=dtype)
    for at, page in (((0, 1), kc.shape[0]), ((1, 0), -1), ((0, 2), 1 << 30)):
        bad = bt.clone()
        bad[at] = page
        o, lse = fa.decode_paged(q, kc, vc, bad, sl, k_exp=ke, v_exp=ve)
        assert status() == fa.FA_ERR_INVALID_ARG
    for lens in ([40, 16 * bt.shape[1] + 1], [-1, 20]):
        bad = torch.tensor(lens, dtype=torch.int32, device="cuda")
        fa.decode_paged(q, kc, vc, bt, bad, k_exp=ke, v_exp=ve)
        assert status() == fa.FA_ERR_INVALID_ARG
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, True)


def test_repeated_captured_and_on_another_stream():
    """The same bits each time; two captured graphs with their own workspaces replayed on two streams
    with lengths that changed after the capture."""
    D, dtype, Hk = 128, torch.bfloat16, 1
    rng = np.random.default_rng(10)
    lens = [2000, 700]
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, True)
    q = randn(2, 8, D, dtype=dtype)
    need = fa.fa_decode_workspace_bytes_ex(2, 8, Hk, D, bt.shape[1])
    assert need > 0
    first, first_lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    for _ in range(3):
        o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
        assert torch.equal(o, first) and torch.equal(lse, first_lse)
    runs = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fa.decode_paged(q, kc, vc, bt, sl, out=o, lse=lse, workspace=ws, k_exp=ke, v_exp=ve)
        runs.append((graph, s, o, lse, ws))
    torch.cuda.synchronize()
    sl.copy_(torch.tensor([1500, 33], dtype=torch.int32))
    torch.cuda.synchronize()
    for graph, s, *_ in runs:
        with torch.cuda.stream(s):
            graph.replay()
    assert status() == fa.FA_OK
    for _, _, o, lse, _ in runs:
        check(o, lse, q, [ks[0][:, :1500], ks[1][:, :33]], [vs[0][:, :1500], vs[1][:, :33]],
              1.0 / math.sqrt(D), dtype, True)


@pytest.mark.parametrize("B,Hk,G,D,q8,width", [
    (72, 1, 2, 128, True, 20), (73, 1, 2, 128, True, 20), (48, 1, 1, 128, False, 20), (49, 1, 1, 128, False, 20),
    (36, 2, 3, 64, False, 20), (9, 8, 8, 64, True, 20), (4, 1, 8, 128, True, 128), (4, 1, 8, 128, True, 129),
    (8, 4, 1, 64, False, 256), (8, 4, 1, 64, False, 257), (31, 1, 4, 64, True, 129), (4, 1, 9, 64, True, 20)])
def test_either_side_of_the_short_step(B, Hk, G, D, q8, width):
    """Sizes at which the step changes its kernel: most units, longest tables, largest groups."""
    rng = np.random.default_rng(B + width)
    lens = [int(x) for x in rng.integers(0, 17 * 16, B)]
    lens[0], lens[-1] = 17 * 16, 0
    if width >= 128:
        lens[1] = 16 * 126 + 5
    dtype = torch.bfloat16
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8)
    bt = widen(bt[:, :-EXTRA] if EXTRA else bt, width - (bt.shape[1] - EXTRA))
    assert bt.shape[1] == width
    q = randn(B, Hk * G, D, dtype=dtype)
    scale = 1.0 / math.sqrt(D)
    o, lse = fa._decode_paged_ex(q, kc, vc, bt, sl, scale, None, None, None, ke, ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, scale, dtype, q8)


def test_many_sequences():
    """More sequences than one launch takes (1024), most of them short, some empty."""
    D, dtype, Hk = 64, torch.float16, 1
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 40, 1500)]
    lens[1023], lens[1024], lens[1499] = 200, 0, 77
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, True)
    q = randn(1500, 2, D, dtype=dtype)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, True)


def test_equal_heads_agree_with_the_plain_step():
    """The grouped kernel on a 16-bit cache with as many heads as queries against decode_paged."""
    D, dtype, lens = 128, torch.float16, [1, 100, 513]
    rng = np.random.default_rng(11)
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, 3, D, dtype, False)
    for c in (kc, vc):  # (the plain step wants finite values in unused slots)
        c.nan_to_num_(0.0)
    q = randn(3, 3, D, dtype=dtype)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl)
    o2, lse2 = fa._decode_paged_ex(q, kc, vc, bt, sl, None, None, None, None, None, None)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)
    check(o2, lse2, q, ks, vs, 1.0 / math.sqrt(D), dtype, False)


def test_serving_steps_from_a_prompt():
    """A prompt written, then tokens one by one: rotary on the query, the rotated key and the value
    appended (e4m3), attention over everything so far; against 64 bits with the held values."""
    D, Hq, Hk, dtype, n0, steps = 64, 8, 2, torch.bfloat16, 21, 14
    freqs, mscale = fa.rotary_freqs(D)
    k, v, q = (randn(2, h, n0 + steps, D, dtype=dtype, seed=i) for i, h in enumerate((Hk, Hk, Hq)))
    rng = np.random.default_rng(12)
    t, pages = tables(rng, [n0 + steps] * 2)
    bt = widen(torch.from_numpy(t).cuda())
    kc, vc, ke, ve = make_cache(pages, Hk, D, dtype, True)
    sl = torch.full((2,), n0, dtype=torch.int32, device="cuda")
    fa.cache_append(k[:, :, :n0], v[:, :, :n0], kc, vc, bt, sl, k_exp=ke, v_exp=ve, freqs=freqs, mscale=mscale)
    for i in range(n0, n0 + steps):
        sl += 1
        fa.cache_append(k[:, :, i:i + 1], v[:, :, i:i + 1], kc, vc, bt, sl, k_exp=ke, v_exp=ve,
                        freqs=freqs, mscale=mscale)
        qr = fa.rotary_apply(q[:, :, i:i + 1], (sl - 1)[:, None], freqs, mscale)
        qr = qr.reshape(2, Hq, D)
        o, lse = fa.decode_paged(qr, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    n = n0 + steps
    hk, hv = held(kc, ke), held(vc, ve)
    pos = np.arange(n)
    ks = [hk[t[b, pos // PAGE], :, pos % PAGE].transpose(1, 0, 2) for b in range(2)]
    vs = [hv[t[b, pos // PAGE], :, pos % PAGE].transpose(1, 0, 2) for b in range(2)]
    check(o, lse, qr, ks, vs, 1.0 / math.sqrt(D), dtype, True)


def test_far_pages_of_a_large_cache():
    """Offsets past 2^32 bytes: the last pages of a cache of 4.5 GB a side."""
    D, Hk, dtype = 128, 8, torch.bfloat16
    pages = (9 << 29) // (Hk * PAGE * D)
    kc = torch.zeros((pages, Hk, PAGE, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.zeros_like(kc.view(torch.uint8)).view(torch.float8_e4m3fn)
    ke = torch.zeros((pages, Hk, PAGE), dtype=torch.uint8, device="cuda")
    ve = torch.zeros_like(ke)
    bt = widen(torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda"))
    sl = torch.tensor([40], dtype=torch.int32, device="cuda")
    k, v = randn(1, Hk, 40, D, dtype=dtype), randn(1, Hk, 40, D, dtype=dtype, seed=1)
    fa.cache_append(k, v, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    q = randn(1, 2 * Hk, D, dtype=dtype, seed=2)
    o, lse = fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    dk, dv = fa.cache_read(kc, vc, bt, sl, 40, k_exp=ke, v_exp=ve, dtype=dtype)
    assert status() == fa.FA_OK
    ks, vs = quantise(gh.f64(k[0]))[0], quantise(gh.f64(v[0]))[0]
    check(o, lse, q, [ks], [vs], 1.0 / math.sqrt(D), dtype, True)
    assert np.array_equal(gh.f64(dk[0]), ks) and np.array_equal(gh.f64(dv[0]), vs)


def test_refusals_of_the_public_call():
    D, Hk = 64, 2
    q = randn(1, 4, D, dtype=torch.bfloat16)
    kc, vc, ke, ve = make_cache(2, Hk, D, torch.bfloat16, True)
    bt = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    sl = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises((ValueError, TypeError)):
        fa.decode_paged(q, kc, vc, bt, sl)                                  # no exponents
    with pytest.raises(ValueError):
        fa.decode_paged(q, kc, vc, bt, sl, k_exp=ke)                        # one of the two
    with pytest.raises(TypeError):
        fa.decode_paged(q, kc, vc, bt.long(), sl, k_exp=ke, v_exp=ve)
    with pytest.raises(ValueError):
        fa.decode_paged(q, kc, vc, bt[:, :1].expand(1, 2), sl.repeat(2), k_exp=ke, v_exp=ve)
    with pytest.raises(ValueError):
        fa.decode_paged(q, kc, vc, bt.cpu(), sl, k_exp=ke, v_exp=ve)
    with pytest.raises(ValueError):
        fa.decode_paged(q.transpose(0, 1), kc, vc, bt, sl, k_exp=ke, v_exp=ve)
    with pytest.raises(fa.FaError):
        fa.decode_paged(q[:, :3].contiguous(), kc, vc, bt, sl, k_exp=ke, v_exp=ve)  # 3 heads on 2
    assert status() == fa.FA_OK
