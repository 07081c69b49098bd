"""The paged cache's writing and reading (fa_cache_append, fa_cache_read) against the definition.

Rows that are not rotated must match bit for bit: a 16-bit cache holds them as they are, an e4m3
cache their one rounding after an exact scaling by a power of two.  Rotated keys differ from the
64-bit rotation by under 1.5e-6 (|x1| + |x2|) mscale (see test_gpu_rotary.py) before the rounding.
"""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_rotary import randn, reference, thetas

pytestmark = pytest.mark.gpu
PAGE = fa.FA_PAGE_TOKENS


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def status():
    torch.cuda.synchronize()
    return fa.fa_get_device_status(torch.cuda.current_stream().cuda_stream)


def quantise(x):
    """(values held, biased exponents) of rows of x (64-bit numpy, finite)."""
    amax = np.abs(x).max(-1)
    m, e = np.frexp(amax)  # amax = m 2^e, 448 = 0.875 * 2^9
    e = np.where(m > 0.875, e - 8, e - 9)
    e = np.where(amax == 0, -127, np.clip(e, -127, 127))
    y = np.ldexp(x, -e[..., None])
    step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
    return np.ldexp(np.round(y / step) * step, e[..., None]), e + 127


def make_cache(pages, H, D, dtype, quant):
    """A cache whose every byte is a NaN pattern: what a call leaves alone must still be there."""
    if quant:
        kc, vc = (torch.full((pages, H, PAGE, D), 0x7F, dtype=torch.uint8, device="cuda")
                  .view(torch.float8_e4m3fn) for _ in range(2))
        ke, ve = (torch.full((pages, H, PAGE), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
        return kc, vc, ke, ve
    return (*(torch.full((pages, H, PAGE, D), math.nan, dtype=dtype, device="cuda") for _ in range(2)),
            None, None)


def held(cache, ex):
    x = cache.float().cpu().double().numpy()
    return x if ex is None else np.ldexp(x, ex.cpu().numpy().astype(int)[..., None] - 127)


def tables(rng, lens, spare=3):
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    total = sum(pages) + spare
    order = rng.permutation(total)
    t = np.zeros((len(lens), max(1, max(pages))), dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        t[b, :n] = order[at:at + n]
        at += n
    return t, total


CASES = [
    # lens (with the new rows), new rows, L, H, D, rotary_dim, interleaved, dtype, quantised
    ([1, 16, 17, 300], [1, 1, 1, 1], 1, 3, 128, 0, False, torch.bfloat16, True),
    ([5, 0, 40], [5, 0, 17], 20, 2, 64, 0, False, torch.float16, True),
    ([64, 33], [64, 30], 64, 1, 128, 128, False, torch.bfloat16, True),
    ([70, 20, 9], [13, 20, 1], 33, 5, 64, 32, True, torch.float16, True),
    ([50], [50], 50, 17, 128, 24, False, torch.bfloat16, True),
    ([3, 100], [3, 100], 100, 2, 128, 0, False, torch.bfloat16, False),
    ([19, 7], [2, 7], 7, 3, 64, 64, False, torch.float16, False),
]


@pytest.mark.parametrize("lens,new,L,H,D,rd,inter,dtype,quant", CASES, ids=lambda x: str(x).replace("torch.", "")[:24])
def test_append_then_read(lens, new, L, H, D, rd, inter, dtype, quant):
    rng = np.random.default_rng(len(lens) * 10 + L)
    B = len(lens)
    t, pages = tables(rng, lens)
    kc, vc, ke, ve = make_cache(pages, H, D, dtype, quant)
    k, v = randn(B, H, L, D, dtype=dtype, seed=L), randn(B, L, H, D, dtype=dtype, seed=L + 1).transpose(1, 2)
    for b in range(B):  # rows behind the new ones are not read
        k[b, :, new[b]:] = math.nan
        v[b, :, new[b]:] = math.inf
    bt, sl, nl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (t, lens, new))
    rot = {}
    if rd:
        freqs, mscale = fa.rotary_freqs(rd)
        th, _ = thetas(rd)
        rot = dict(freqs=freqs, mscale=mscale, interleaved=inter)
    fa.cache_append(k, v, kc, vc, bt, sl, nl, k_exp=ke, v_exp=ve, **rot)
    n = max(lens) + 5
    dk, dv = fa.cache_read(kc, vc, bt, sl, n, k_exp=ke, v_exp=ve, dtype=dtype)
    assert status() == fa.FA_OK
    hk, hv = held(kc, ke), held(vc, ve)
    written = np.zeros((pages, PAGE), dtype=bool)
    for b in range(B):
        start = lens[b] - new[b]
        pos = np.arange(start, lens[b])
        pg, sl_ = t[b, pos // PAGE], pos % PAGE
        written[pg, sl_] = True
        for name, x, h, ex in (("k", k, hk, ke), ("v", v, hv, ve)):
            rows = gh.f64(x[b, :, :new[b]])  # [H, n, D]
            got = h[pg, :, sl_].transpose(1, 0, 2)
            if name == "k" and rd:
                ref, mag = reference(x[b:b + 1, :, :new[b]], pos[None], th, 1.0, inter)
                ref, slack = ref[0], 1.5e-6 * mag[0]
                if quant:
                    _, e = quantise(ref)
                    # half a step of the row's grid: 2^-4 of the value, 2^-10 2^e near zero; the
                    # exponent may be one higher where the largest value is next to the border
                    bound = np.maximum(2.0 ** -4 * np.abs(ref), np.ldexp(1.0, e - 127 - 9)[..., None]) + 1.1 * slack
                else:
                    half = torch.finfo(dtype).eps / 2
                    bound = half * np.abs(ref) + 1.1 * slack + 2.0 ** -25
                assert np.all(np.abs(got - ref) <= bound)
            elif quant:
                ref, e = quantise(rows)
                assert np.array_equal(got, ref)
                assert np.array_equal(ex.cpu().numpy()[pg, :, sl_].T, e)
            else:
                assert np.array_equal(got, rows)
        # what reading returns: the held rows, then zeros (the unwritten slots hold NaN)
        for d, h in ((dk, hk), (dv, hv)):
            all_pos = np.arange(lens[b])
            want = torch.from_numpy(h[t[b, all_pos // PAGE], :, all_pos % PAGE].transpose(1, 0, 2)).to(dtype)
            assert torch.equal(d[b, :, :lens[b]].cpu().nan_to_num(7.0), want.nan_to_num(7.0))
            assert not torch.any(d[b, :, lens[b]:])
    assert np.all(np.isnan(hk.transpose(0, 2, 1, 3)[~written]))  # other slots as they were
    assert np.all(np.isnan(hv.transpose(0, 2, 1, 3)[~written]))


def test_append_token_by_token_equals_one_prefill():
    """A prompt written at once and the same tokens written one by one give the same cache."""
    H, D, n = 2, 128, 37
    t = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    k, v = randn(1, H, n, D, dtype=torch.bfloat16), randn(1, H, n, D, dtype=torch.bfloat16, seed=1)
    freqs, m = fa.rotary_freqs(D)
    caches = [make_cache(3, H, D, torch.bfloat16, True) for _ in range(2)]
    for c in caches:
        for x in c:
            x.view(torch.uint8).zero_()
    one, many = caches
    fa.cache_append(k, v, one[0], one[1], t, torch.tensor([n], dtype=torch.int32, device="cuda"),
                    k_exp=one[2], v_exp=one[3], freqs=freqs, mscale=m)
    for i in range(n):
        fa.cache_append(k[:, :, i:i + 1], v[:, :, i:i + 1], many[0], many[1], t,
                        torch.tensor([i + 1], dtype=torch.int32, device="cuda"),
                        k_exp=many[2], v_exp=many[3], freqs=freqs, mscale=m)
    assert status() == fa.FA_OK
    for a, b in zip(one, many):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_quantised_extremes():
    """Rows of zeros, of the smallest and the largest values, borders of the exponent, ties, and
    rows with an infinity or a NaN."""
    D, H = 64, 1
    rows = torch.zeros((12, D), dtype=torch.float32)
    rows[1, 3] = 2.0 ** -133                      # a bf16 subnormal: below the smallest scale
    rows[2, :] = 2.0 ** -126
    rows[3, 0] = torch.finfo(torch.bfloat16).max
    rows[3, 1] = 1.0                              # under half the row's smallest step: 0
    rows[4, 0], rows[4, 1] = 448.0, 449.0 / 2     # exactly the border
    rows[5, 0], rows[5, 1] = 450.0, 1.0           # just past it (bf16: 450)
    rows[6, :8] = torch.tensor([448, 17, 18, 19, 34, 38, 2.0 ** -10, 3 * 2.0 ** -10])  # ties
    rows[7, 2], rows[8, 2], rows[9, 2] = math.inf, -math.inf, math.nan
    rows[7, 1] = 3.0
    rows[10, :] = -0.0
    rows[11, :] = torch.linspace(-5, 5, D)
    x = rows.to(torch.bfloat16).cuda()[None, None]
    kc, vc, ke, ve = make_cache(1, H, D, torch.bfloat16, True)
    t = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    n = torch.tensor([12], dtype=torch.int32, device="cuda")
    fa.cache_append(x, x, kc, vc, t, n, k_exp=ke, v_exp=ve)
    k, v = fa.cache_read(kc, vc, t, n, 12, k_exp=ke, v_exp=ve, dtype=torch.bfloat16)
    assert status() == fa.FA_OK
    xs = gh.f64(x[0, 0])
    for r in range(12):
        for d, ex in ((k, ke), (v, ve)):
            if r in (7, 8, 9):
                assert int(ex[0, 0, r]) == 255 and torch.isnan(d[0, 0, r]).all()
                continue
            ref, e = quantise(xs[r])
            assert int(ex[0, 0, r]) == e, r
            # reading rounds to bf16: exact but for the largest value, held as 256 * 2^120 = 2^128,
            # which has no finite bf16
            assert np.array_equal(gh.f64(d[0, 0, r]), gh.f64(torch.from_numpy(ref).to(torch.bfloat16))), r


def test_append_and_read_report_bad_device_data():
    H, D = 2, 64
    k = randn(2, H, 4, D, dtype=torch.float16)
    good = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cases = [
        (torch.tensor([[0, 1], [2, 4]], dtype=torch.int32, device="cuda"), i32(4, 20), None),  # page 4 of 4
        (torch.tensor([[0, 1], [-1, 3]], dtype=torch.int32, device="cuda"), i32(4, 4), None),
        (good, i32(4, 33), None),             # longer than the table
        (good, i32(4, 3), None),              # shorter than the rows it adds
        (good, i32(4, -1), i32(4, 0)),
        (good, i32(4, 9), i32(4, 5)),         # more rows than k has
        (good, i32(4, 9), i32(4, -2)),
    ]
    for bt, sl, nl in cases:
        kc, vc, ke, ve = make_cache(4, H, D, torch.float16, True)
        fa.cache_append(k, k, kc, vc, bt, sl, nl, k_exp=ke, v_exp=ve)
        assert status() == fa.FA_ERR_INVALID_ARG
        assert torch.isnan(kc[2:].float()).all() and not torch.isnan(kc[0, :, :4].float()).any()
        assert status() == fa.FA_OK
    kc, vc, ke, ve = make_cache(4, H, D, torch.float16, True)
    ke.fill_(127), ve.fill_(127)
    kc.view(torch.uint8).fill_(0x38), vc.view(torch.uint8).fill_(0x38)  # ones
    for bt, sl in ((cases[0][0], i32(4, 20)), (good, i32(4, 33)), (good, i32(4, -5))):
        dk, _ = fa.cache_read(kc, vc, bt, sl, 32, k_exp=ke, v_exp=ve, dtype=torch.float16)
        assert status() == fa.FA_ERR_INVALID_ARG
        assert torch.all(dk[0, :, :4] == 1) and not torch.any(dk[1, :, 16:])


def test_unused_places_of_a_batch_and_empty_calls():
    H, D = 1, 64
    kc, vc, ke, ve = make_cache(2, H, D, torch.bfloat16, True)
    t = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    k = randn(2, H, 1, D, dtype=torch.bfloat16)
    sl = torch.tensor([1, 0], dtype=torch.int32, device="cuda")  # the second place is unused
    fa.cache_append(k, k, kc, vc, t, sl, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    assert torch.isnan(kc[1].float()).all() and torch.isnan(kc[0, :, 1:].float()).all()
    assert not torch.isnan(kc[0, :, 0].float()).any()
    fa.cache_append(k[:, :, :0], k[:, :, :0], kc, vc, t, sl, k_exp=ke, v_exp=ve)
    fa.cache_append(k[:0], k[:0], kc, vc, t[:0], sl[:0], k_exp=ke, v_exp=ve)
    a, _ = fa.cache_read(kc, vc, t, sl, 0, k_exp=ke, v_exp=ve, dtype=torch.bfloat16)
    assert a.shape == (2, H, 0, D) and status() == fa.FA_OK


def test_read_back_continues_a_prompt():
    """A prompt in two chunks over an e4m3 cache: the second chunk's queries attend to the rows
    read back (Lk > Lq) and get what attention over the held values gives in 64 bits."""
    import oracle
    H, D, n0, n1 = 2, 64, 45, 30
    n = n0 + n1
    q, k, v = (randn(1, H, n, D, dtype=torch.bfloat16, seed=i) for i in range(3))
    kc, vc, ke, ve = make_cache(8, H, D, torch.bfloat16, True)
    t = torch.tensor([[5, 1, 7, 2, 0]], dtype=torch.int32, device="cuda")
    for a, b in ((0, n0), (n0, n)):
        sl = torch.tensor([b], dtype=torch.int32, device="cuda")
        fa.cache_append(k[:, :, a:b], v[:, :, a:b], kc, vc, t, sl, k_exp=ke, v_exp=ve)
    dk, dv = fa.cache_read(kc, vc, t, sl, n, k_exp=ke, v_exp=ve, dtype=torch.bfloat16)
    o, _ = fa.forward(q[:, :, n0:], dk, dv, causal=True)
    assert status() == fa.FA_OK
    ref, _ = oracle.forward(gh.f64(q[:, :, n0:]), quantise(gh.f64(k))[0], quantise(gh.f64(v))[0],
                            1.0 / math.sqrt(D), True)
    err = gh.o_errors(gh.f64(o), ref, torch.bfloat16)
    assert err["o_max"] <= gh.O_MAX_ABS and err["o_mean"] <= gh.O_MEAN_ABS, err
