"""Grouped decode of 2048 (sequence, cache head, query block) units and more in one launch, whose pages
are dealt out in three rounds where there are 16 a worker, against the definition in 64 bits (every
row; tolerances of test_gpu_decode_gqa.py).

Each case says whether its line of pages is long enough for three rounds, by the split's own rule, so
that a case which no longer reaches it fails."""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import tiled_attention_08_gb300 as fa
from test_gpu_cache import PAGE, make_cache, quantise, status, tables
from test_gpu_decode_gqa import check
from test_gpu_rotary import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gh.require_gpu()


def fill(rng, lens, Hk, D, dtype, q8, long=3000):
    """As in test_gpu_decode_gqa.py, sequences of `long` tokens and more written one by one (a dense
    batch as long as the longest would not fit)."""
    t, pages = tables(rng, lens)
    kc, vc, ke, ve = make_cache(pages, Hk, D, dtype, q8)
    bt, sl = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    rows = [[None] * len(lens), [None] * len(lens)]
    short = [b for b, n in enumerate(lens) if n < long]
    for group in [short] + [[b] for b, n in enumerate(lens) if n >= long]:
        at = torch.tensor(group, device="cuda")
        n = sl[at].contiguous()
        L = max(1, int(n.max()))
        k = randn(len(group), Hk, L, D, dtype=dtype, seed=group[0])
        v = randn(len(group), Hk, L, D, dtype=dtype, seed=group[0] + 5000)
        fa.cache_append(k, v, kc, vc, bt[at].contiguous(), n, n, k_exp=ke, v_exp=ve)
        for r, x in zip(rows, (k, v)):
            for i, b in enumerate(group):
                held = gh.f64(x[i, :, :lens[b]])
                r[b] = quantise(held)[0] if q8 and lens[b] else held
    return kc, vc, ke, ve, bt, sl, rows[0], rows[1]


def three_rounds(lens, Hk, group, D, q8):
    """The rule of the split (fa_decode_gqa.cu) for these lengths."""
    q_rows = 8 if group <= 8 else 16
    per_seq = Hk * -(-group // q_rows)
    units = len(lens) * per_seq
    per_sm = 4 * (3 if group > 8 or (D == 128 and not q8) else 4)
    total = sum(-(-n // PAGE) for n in lens) * per_seq
    workers = max(1, min(total if total <= 1024 else total // 4, 128 * units, 152 * per_sm))
    return units >= 2048 and total >= 16 * workers


def mixed(seed, B, hi, extra):
    """Empty, one-token, page-long and longer sequences; `extra`: {place: length}."""
    r = np.random.default_rng(seed)
    lens = [int(x) for x in r.integers(0, hi, B)]
    for i, n in enumerate((0, 1, 15, 16, 17, 0, 0)):
        lens[(7 * i) % B] = n
    for at, n in extra.items():
        lens[at] = n
    return lens


CASES = {
    # lens, cache heads, group, D, dtype, e4m3, reaches three rounds
    "e4m3_128": (mixed(1, 64, 700, {20: 6000, 63: 2500}), 32, 1, 128, torch.bfloat16, True, True),
    "e4m3_64": (mixed(2, 64, 900, {0: 4000, 33: 0}), 32, 2, 64, torch.float16, True, True),
    "16bit_128": (mixed(3, 64, 700, {61: 5000}), 32, 1, 128, torch.bfloat16, False, True),
    "16bit_64": (mixed(4, 70, 800, {}), 32, 2, 64, torch.float16, False, True),
    "ends_empty": (mixed(5, 100, 600, {98: 0, 99: 0, 0: 0}), 32, 1, 64, torch.bfloat16, True, True),
    "group_9": (mixed(6, 64, 700, {}), 32, 9, 64, torch.bfloat16, True, True),
    "group_20": (mixed(7, 128, 900, {}), 8, 20, 128, torch.float16, False, True),
    # One unit reaches from the first round through the second into the third, on either cache.
    "across_e4m3": (mixed(8, 1024, 96, {1023: 262144}), 2, 1, 64, torch.bfloat16, True, True),
    "across_16bit": (mixed(9, 1024, 96, {1023: 262144}), 2, 1, 64, torch.float16, False, True),
    "across_both": (mixed(10, 1024, 96, {600: 150000, 1000: 120000}), 2, 1, 64, torch.bfloat16, True, True),
    # 2048 units whose pages are too few: one round.
    "mostly_empty": ([0] * 60 + [40, 0, 1, 300], 32, 1, 128, torch.bfloat16, True, False),
    "short": (mixed(11, 256, 20, {}), 8, 4, 64, torch.float16, False, False),
    "none": ([0] * 64, 32, 1, 64, torch.bfloat16, True, False),
}


@pytest.mark.parametrize("name", CASES)
def test_rows_of_many_units(name):
    lens, Hk, group, D, dtype, q8, three = CASES[name]
    assert three_rounds(lens, Hk, group, D, q8) == three
    rng = np.random.default_rng(len(lens))
    kc, vc, ke, ve, bt, sl, ks, vs = fill(rng, lens, Hk, D, dtype, q8)
    q = randn(len(lens), Hk * group, D, dtype=dtype, seed=3)
    # What the workspace held before, and how often the step has run, must not matter.
    ws = torch.full((fa.fa_decode_workspace_bytes_ex(len(lens), Hk * group, Hk, D, bt.shape[1]),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    o, lse = fa._decode_paged_ex(q, kc, vc, bt, sl, workspace=ws, k_exp=ke, v_exp=ve)
    assert status() == fa.FA_OK
    check(o, lse, q, ks, vs, 1.0 / math.sqrt(D), dtype, q8)
    for _ in range(2):
        o2, lse2 = fa._decode_paged_ex(q, kc, vc, bt, sl, workspace=ws, k_exp=ke, v_exp=ve)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,Hk,group,D,dtype", [
    (mixed(12, 64, 700, {5: 4000}), 32, 1, 128, torch.bfloat16),
    (mixed(13, 256, 700, {255: 0}), 8, 4, 64, torch.float16),
    (mixed(14, 1030, 96, {1000: 262144, 1029: 50}), 2, 1, 64, torch.bfloat16),  # and a second, short launch
], ids=["128", "64", "across"])
def test_behind_a_shared_prefix(lens, Hk, group, D, dtype):
    assert three_rounds(lens[:1024], Hk, group, D, False)
    prefix = 333
    rng = np.random.default_rng(D)
    kc, vc, _, _, bt, sl, ks, vs = fill(rng, [prefix] + lens, Hk, D, dtype, False)
    q = randn(len(lens), Hk * group, D, dtype=dtype, seed=4)
    pt = bt[0, :-(-prefix // PAGE)].contiguous()
    own = bt[1:].contiguous()
    o, lse = fa.decode_shared_prefix(q, kc, vc, pt, prefix, own, sl[1:].contiguous())
    assert status() == fa.FA_OK
    check(o, lse, q, [np.concatenate((ks[0], k), 1) for k in ks[1:]],
          [np.concatenate((vs[0], v), 1) for v in vs[1:]], 1.0 / math.sqrt(D), dtype, False)
    o2, lse2 = fa.decode_shared_prefix(q, kc, vc, pt, prefix, own, sl[1:].contiguous())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
