"""Argument checks of the rotary, cache and grouped decode calls on the host (no GPU work).

Every call here is refused, or has nothing to do, before the library touches the CUDA runtime.
"""
import math

import pytest

import tiled_attention_08_gb300 as fa

A = 0x100000  # fake, 16-byte aligned device addresses: never dereferenced by these calls
MB = 1 << 20
BAD, UNS, OK = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tiled_attention_08_gb300 import build
    build.build()
    return fa.load_library()


def _rotary(B=2, Hq=2, Hk=1, L=16, D=64, rd=64, mscale=1.0, inter=0, inverse=0, dtype=0, pstride=16,
            strides=None, **ptrs):
    p = dict(q=A, k=A + MB, qo=A + 2 * MB, ko=A + 3 * MB, pos=A + 4 * MB, freqs=A + 5 * MB)
    p.update(ptrs)
    sq, sk = (Hq * L * D, L * D, D), (Hk * L * D, L * D, D)
    return fa.fa_rotary(p["q"], p["k"], p["qo"], p["ko"], strides or [sq, sk, sq, sk], p["pos"],
                        pstride, p["freqs"], rd, mscale, inter, inverse, B, Hq, Hk, L, D, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), BAD),
    (dict(B=-1), BAD),
    (dict(Hk=-1), BAD),
    (dict(L=-1), BAD),
    (dict(D=0), BAD),
    (dict(D=96), UNS),
    (dict(rd=0), BAD),
    (dict(rd=63), BAD),
    (dict(rd=66), BAD),
    (dict(rd=-2), BAD),
    (dict(mscale=math.nan), BAD),
    (dict(mscale=math.inf), BAD),
    (dict(inter=2), BAD),
    (dict(inverse=-1), BAD),
    (dict(q=0), BAD),
    (dict(ko=0), BAD),
    (dict(freqs=0), BAD),
    (dict(freqs=A + 5 * MB + 4), BAD),           # freqs not 8-byte aligned
    (dict(pos=A + 4 * MB + 2), BAD),
    (dict(pstride=-1), BAD),
    (dict(q=A + 8), BAD),                        # misaligned
    (dict(qo=A + 1024), BAD),                    # inside q, but not q itself
    (dict(ko=A), BAD),                           # k's output on q
    (dict(ko=A + 2 * MB + 2048), BAD),           # the outputs overlap
    (dict(qo=A + 4 * MB), BAD),                  # on the positions
    (dict(strides=[(2048, 1024, 60)] * 4), BAD),
    (dict(strides=[(2048, 0, 64)] * 4), BAD),    # zero head stride with two heads
    (dict(B=1 << 20, L=1 << 12), UNS),
    (dict(Hq=65535, Hk=1, B=1, L=1), UNS),
    (dict(B=0), OK),
    (dict(L=0, q=0, k=0, qo=0, ko=0, freqs=0), OK),
    (dict(Hq=0, Hk=0), OK),
], ids=lambda x: str(x)[:48])
def test_rotary_argument_checks(kw, status):
    assert _rotary(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), OK),
    (dict(scaling=3, factor=16.0, orig=4096.0), OK),
    (dict(rd=0), BAD),
    (dict(rd=7), BAD),
    (dict(base=0.5), BAD),
    (dict(base=math.inf), BAD),
    (dict(base=math.nan), BAD),
    (dict(scaling=4), BAD),
    (dict(scaling=-1), BAD),
    (dict(scaling=1, factor=0.5), BAD),
    (dict(scaling=1, factor=math.nan), BAD),
    (dict(scaling=3, factor=2.0), BAD),          # needs the trained length
    (dict(scaling=3, factor=2.0, orig=math.inf), BAD),
    (dict(scaling=2, factor=2.0, rd=2), BAD),    # exponent rd / (rd - 2)
    (dict(scaling=2, factor=1e300, rd=4), BAD),  # the grown base overflows
], ids=lambda x: str(x)[:48])
def test_rotary_freqs_checks(kw, status):
    kw = dict(dict(rd=64, base=10000.0, scaling=0, factor=1.0, orig=0.0), **kw)
    assert fa.fa_rotary_freqs(kw["rd"], kw["base"], kw["scaling"], kw["factor"], kw["orig"])[0] == status


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rotary_freqs_values(scaling):
    """Turns per position of every form, in 64-bit fixed point."""
    rd, base, f, orig = 64, 10000.0, 8.0, 2048.0
    st, freqs, mscale = fa.fa_rotary_freqs(rd, base, fa.FA_ROTARY_SCALING[scaling], f, orig)
    assert st == OK and len(freqs) == rd // 2
    for i, w in enumerate(freqs):
        b = base * f ** (rd / (rd - 2)) if scaling == "ntk" else base
        th = b ** (-2 * i / rd)
        if scaling == "linear":
            th /= f
        if scaling == "yarn":
            keep = min(1.0, max(0.0, (orig * th / (2 * math.pi) - 1) / 31))
            th = th * keep + th / f * (1 - keep)
        # pow and the quotient are each within a step or two of 2^-53; the fixed point rounds to
        # a whole number of 2^-64 turns, off by half of one: 2 pi 2^-65 radians
        assert abs(w / 2.0 ** 64 * 2 * math.pi - th) <= th * 2.0 ** -49 + 2 * math.pi * 2.0 ** -65, i
    assert abs(mscale - (0.1 * math.log(f) + 1 if scaling == "yarn" else 1.0)) <= 2.0 ** -23
    with pytest.raises(ValueError):
        fa.rotary_freqs(64, scaling="cubic", device="cpu")
    with pytest.raises(fa.FaError):
        fa.rotary_freqs(65, device="cpu")
    table, _ = fa.rotary_freqs(rd, base, scaling, f, orig, device="cpu")
    assert table.tolist() == freqs


def _append(B=2, H=2, L=4, D=64, rd=0, pages=8, maxp=4, dtype=0, cdtype=1, **ptrs):
    p = dict(k=A, v=A + MB, kc=A + 2 * MB, vc=A + 3 * MB, ke=A + 4 * MB, ve=A + 5 * MB, bt=A + 6 * MB,
             sl=A + 7 * MB, nl=A + 8 * MB, freqs=A + 9 * MB, st=None)
    p.update(ptrs)
    c = (H * L * D, L * D, D)
    return fa.fa_cache_append(p["k"], p["v"], p["st"] or [c, c], p["kc"], p["vc"], p["ke"], p["ve"],
                              p["bt"], p["sl"], p["nl"], p["freqs"], rd, 1.0, 0, B, H, L, D, pages, maxp,
                              dtype, cdtype, None)


def _read(B=2, H=2, L=4, D=64, pages=8, maxp=4, dtype=0, cdtype=1, **ptrs):
    p = dict(k=A, v=A + MB, kc=A + 2 * MB, vc=A + 3 * MB, ke=A + 4 * MB, ve=A + 5 * MB, bt=A + 6 * MB,
             sl=A + 7 * MB, st=None)
    p.update(ptrs)
    c = (H * L * D, L * D, D)
    return fa.fa_cache_read(p["kc"], p["vc"], p["ke"], p["ve"], p["bt"], p["sl"], p["k"], p["v"],
                            p["st"] or [c, c], B, H, L, D, pages, maxp, dtype, cdtype, None)


COMMON = [
    (dict(dtype=7), BAD),
    (dict(cdtype=2), BAD),
    (dict(B=-1), BAD),
    (dict(L=-1), BAD),
    (dict(pages=-1), BAD),
    (dict(D=0), BAD),
    (dict(D=80), UNS),
    (dict(B=65536), UNS),
    (dict(H=65536), UNS),
    (dict(maxp=1 << 28), UNS),                   # 16 * max_pages past 31 bits
    (dict(L=(1 << 31) - 1), UNS),                # the last tile's rows past 31 bits
    (dict(k=0), BAD),
    (dict(v=A + MB + 2), BAD),
    (dict(kc=0), BAD),
    (dict(ke=0), BAD),
    (dict(bt=0), BAD),
    (dict(sl=0), BAD),
    (dict(sl=A + 7 * MB + 1), BAD),
    (dict(st=[(512, 256, 65)] * 2), BAD),
    (dict(st=[(512, -256, 64)] * 2), BAD),
    (dict(kc=A + 512), BAD),                     # the cache on the rows
    (dict(v=A + 4 * MB), BAD),                   # the rows on the exponents
    (dict(L=0, k=0, v=0), OK),
    (dict(B=0), OK),
    (dict(H=0), OK),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(rd=3), BAD),
    (dict(rd=66), BAD),
    (dict(rd=64, freqs=0), BAD),
    (dict(nl=A + 8 * MB + 2), BAD),
    (dict(vc=A + 2 * MB + 4096), BAD),           # the two caches overlap
    (dict(ve=A + 3 * MB), BAD),                  # exponents on the value cache
    (dict(bt=A + 2 * MB), BAD),                  # the table inside the cache
], ids=lambda x: str(x)[:48])
def test_append_argument_checks(kw, status):
    assert _append(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(v=A + 256), BAD),                      # the outputs overlap
], ids=lambda x: str(x)[:48])
def test_read_argument_checks(kw, status):
    assert _read(**kw) == status


def _decode(B=2, Hq=4, Hk=2, D=64, pages=8, maxp=4, scale=0.125, dtype=0, cdtype=1, ws_bytes=1 << 20, **ptrs):
    p = dict(q=A, kc=A + MB, vc=A + 2 * MB, ke=A + 3 * MB, ve=A + 4 * MB, bt=A + 5 * MB, sl=A + 6 * MB,
             o=A + 7 * MB, lse=A + 8 * MB, ws=A + 9 * MB)
    p.update(ptrs)
    return fa.fa_decode_paged_ex(p["q"], p["kc"], p["vc"], p["ke"], p["ve"], p["bt"], p["sl"], p["o"],
                                 p["lse"], p["ws"], ws_bytes, B, Hq, Hk, D, pages, maxp, scale, dtype,
                                 cdtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), BAD),
    (dict(cdtype=-1), BAD),
    (dict(D=96), UNS),
    (dict(D=-64), BAD),
    (dict(Hq=-1), BAD),
    (dict(Hq=5), BAD),                           # not a multiple of Hk
    (dict(Hk=0), BAD),
    (dict(scale=math.nan), BAD),
    (dict(B=65536), UNS),
    (dict(Hq=65536 * 20, Hk=65536), UNS),
    (dict(Hq=1 << 20, Hk=4, B=1 << 12), UNS),
    (dict(B=1, Hq=65535, Hk=65535, maxp=(1 << 27) - 1), UNS),  # a warp's pages past 31 bits
    (dict(q=0), BAD),
    (dict(lse=0), BAD),
    (dict(ve=0), BAD),
    (dict(kc=A + MB + 8), BAD),
    (dict(ke=A + 3 * MB + 8), BAD),
    (dict(bt=0), BAD),
    (dict(o=A + MB), BAD),                       # o inside the key cache
    (dict(lse=A + 7 * MB + 64), BAD),            # lse overlaps o
    (dict(o=A + 3 * MB), BAD),                   # o on the exponents
    (dict(B=1, Hq=1, Hk=1, maxp=64, ws_bytes=16), BAD),
    (dict(B=1, Hq=1, Hk=1, maxp=64, ws=0), BAD),
    (dict(B=1, Hq=1, Hk=1, maxp=64, ws=A + 7 * MB), BAD),
    (dict(B=0), OK),
    (dict(Hq=0), OK),
], ids=lambda x: str(x)[:48])
def test_grouped_decode_argument_checks(kw, status):
    assert _decode(**kw) == status


def test_grouped_decode_workspace():
    """8 bytes a unit, then two slots of the group's rows (16 at most) for every warp of a step."""
    def need(B, Hq, Hk, D, max_pages):
        g = Hq // Hk
        q_rows = 8 if g <= 8 else 16
        chunk = min(B, 1024)
        units = chunk * Hk * -(-g // q_rows)
        ctas = min(4 * 152, max(1, -(-units * max_pages // 4)))
        up = lambda n: (n + 15) // 16 * 16  # noqa: E731
        slots = 2 * 4 * ctas * min(g, q_rows) * (3 if units >= 2048 else 1)
        return up(8 * units) + up(slots * D * 4) + up(slots * 4)

    for args in ((256, 32, 8, 128, 256), (1, 8, 1, 128, 16), (1, 8, 1, 128, 1024), (5, 40, 2, 64, 9),
                 (2, 4, 2, 64, 0), (3000, 2, 2, 64, 1), (256, 32, 32, 128, 256), (255, 64, 8, 64, 9)):
        assert fa.fa_decode_workspace_bytes_ex(*args) == need(*args), args
    assert fa.fa_decode_workspace_bytes_ex(1, 8, 3, 128, 1024) == 0     # invalid
    assert fa.fa_decode_workspace_bytes_ex(1, 8, 1, 96, 1024) == 0
    assert fa.fa_decode_workspace_bytes_ex(-1, 8, 1, 64, 1024) == 0


@pytest.mark.parametrize("lens,per_seq,warps,rounds", [
    ([333], 8, 44, 1), ([0, 0, 5], 1, 4, 1), ([0], 3, 4, 1), ([1] * 40, 2, 20, 1),
    ([7, 0, 4096, 16, 1], 3, 2432, 1), ([16384, 100], 1, 516, 1), (list(range(300)), 4, 2432, 1),
    (list(range(300)), 40, 24, 3), ([1, 0, 5000, 17, 64], 8, 12, 3), ([3] * 500, 4, 8, 3),
    ([17] * 40, 2, 8, 3)])
def test_grouped_decode_split_model(lens, per_seq, warps, rounds):
    """The decode kernel's split as its comment states it: every page in one stretch, at most one
    part of a warp that began before it and one that ends behind it, and the first warp and the
    number that a unit's first warp notes for the merge those that left its parts."""
    pages = [-(-n // 16) for n in lens]
    cum = [0]
    for n in pages:
        cum.append(cum[-1] + n)
    total = cum[-1] * per_seq
    workers = max(1, min(total if total <= 1024 else total // 4, 128 * len(lens) * per_seq, warps))
    if total < 16 * workers:
        rounds = 1
    at = [0, total // 64 * 52, total // 64 * 60, total] if rounds == 3 else [0, total]

    def start(r, i):
        return at[r] + (at[r + 1] - at[r]) * i // workers

    def worker_of(x):
        r = 0
        while r + 1 < rounds and x >= at[r + 1]:
            r += 1
        return r * workers + ((x - at[r] + 1) * workers - 1) // (at[r + 1] - at[r])

    left, noted = {}, {}
    seen = 0
    for w in range(workers * rounds if total else 0):
        x0, end = start(w // workers, w % workers), start(w // workers, w % workers + 1)
        x, slots = x0, set()
        while x < end:
            b = max(i for i in range(len(lens)) if cum[i] * per_seq <= x and pages[i])
            unit, pg = divmod(x - cum[b] * per_seq, pages[b])
            stop = min(end, x + pages[b] - pg)
            slot = None
            if pg > 0 or stop - x < pages[b]:
                slot = 2 * w + (0 if pg > 0 else 1)
                assert slot not in slots
                slots.add(slot)
            if pg == 0:
                last = x + pages[b] - 1
                noted[b, unit] = (w, 1 if last < end else worker_of(last) - w + 1)
            left.setdefault((b, unit), []).append((w, slot))
            seen += stop - x
            x = stop
    assert seen == total
    for b in range(len(lens)):
        for unit in range(per_seq):
            if not pages[b]:
                assert (b, unit) not in left
                continue
            w0, n = noted[b, unit]
            if n == 1:
                assert left[b, unit] == [(w0, None)]
            else:
                assert left[b, unit] == [(w, 2 * w + (1 if w == w0 else 0)) for w in range(w0, w0 + n)]


def _prefix(B=2, Hq=4, Hk=2, D=64, prefix=100, pages=8, maxp=4, scale=0.125, dtype=0, ws_bytes=1 << 20, **ptrs):
    p = dict(q=A, kc=A + MB, vc=A + 2 * MB, pt=A + 3 * MB, bt=A + 5 * MB, sl=A + 6 * MB, o=A + 7 * MB,
             lse=A + 8 * MB, ws=A + 9 * MB)
    p.update(ptrs)
    return fa.fa_decode_shared_prefix(p["q"], p["kc"], p["vc"], p["pt"], prefix, p["bt"], p["sl"], p["o"],
                                      p["lse"], p["ws"], ws_bytes, B, Hq, Hk, D, pages, maxp, scale, dtype,
                                      None)


@pytest.mark.parametrize("kw,status", [
    (dict(prefix=-1), BAD),
    (dict(prefix=(1 << 31) - 1), UNS),
    (dict(dtype=2), BAD),
    (dict(D=72), UNS),
    (dict(Hq=3), BAD),
    (dict(Hq=129, Hk=1), UNS),                   # more rows of one sequence than a query tile
    (dict(scale=math.inf), BAD),
    (dict(q=A + 4), BAD),
    (dict(o=0), BAD),
    (dict(kc=0), BAD),
    (dict(pt=0), BAD),
    (dict(pt=A + 3 * MB + 2), BAD),
    (dict(pages=0), BAD),                        # a prefix, but no page
    (dict(ws=0), BAD),
    (dict(ws_bytes=64), BAD),
    (dict(ws=A + 9 * MB + 8), BAD),
    (dict(ws=A + 3 * MB - 64), BAD),             # the workspace on the prefix's table
    (dict(o=A + 2 * MB + 1024), BAD),            # o inside the value cache
    (dict(B=0), OK),
], ids=lambda x: str(x)[:48])
def test_shared_prefix_argument_checks(kw, status):
    assert _prefix(**kw) == status


def test_shared_prefix_workspace():
    ws = fa.fa_shared_prefix_workspace_bytes
    base = fa.fa_decode_workspace_bytes_ex(2, 4, 2, 64, 4)
    assert ws(2, 4, 2, 64, 0, 4) == base
    # with a prefix: the rows' own part, and one part for one key tile, two for two
    assert ws(2, 4, 2, 64, 100, 4) == base + 2 * (2 * 4 * 65 * 4)
    assert ws(2, 4, 2, 64, 200, 4) == base + 3 * (2 * 4 * 65 * 4)
    assert ws(2, 4, 2, 64, -1, 4) == 0
    assert ws(2, 130, 1, 64, 100, 4) == 0
    # every part a CTA can write has a place: all stretches of all sizes
    for Hk, pairs_b, tiles in ((1, 1, 200), (2, 40, 77), (8, 300, 31), (32, 256, 128), (3, 513, 5)):
        rows_b = min(128, pairs_b)
        n_pairs = ((pairs_b + rows_b - 1) // rows_b + 1) // 2
        units = Hk * n_pairs * tiles
        grid = min(152, max((units + 3) // 4, min(units, 38)))
        first = [units * c // grid for c in range(grid + 1)]
        most = 0
        for item in range(Hk * n_pairs):
            lo, hi = item * tiles, (item + 1) * tiles
            ctas = [c for c in range(grid) if first[c] < hi and first[c + 1] > lo]
            assert ctas[0] == ((lo + 1) * grid - 1) // units
            most = max(most, len(ctas))
        rows = pairs_b * Hk * 65 * 4
        parts = (ws(pairs_b, Hk, Hk, 64, tiles * 128, 0) - ws(pairs_b, Hk, Hk, 64, 0, 0)) // rows - 1
        assert most <= parts <= tiles, (Hk, pairs_b, tiles, most, parts)
