"""Argument checks of the sliding-window calls on the host (no GPU work).

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


def strides(H, L, D):
    return H * L * D, L * D, D


def _fwd(B=2, Hq=4, Hk=2, Lq=32, Lk=64, D=64, window=8, sinks=1, scale=0.125, dtype=0, st=None, **ptrs):
    p = dict(q=A, k=A + MB, v=A + 2 * MB, o=A + 3 * MB, lse=A + 4 * MB)
    p.update(ptrs)
    q, k = strides(Hq, Lq, D), strides(Hk, Lk, D)
    return fa.fa_window_fwd(p["q"], p["k"], p["v"], p["o"], p["lse"], st or [q, k, k, q], B, Hq, Hk, Lq, Lk, D,
                            window, sinks, scale, dtype, None)


def _bwd(B=2, Hq=4, Hk=2, Lq=32, Lk=64, D=64, window=8, sinks=1, scale=0.125, dtype=0, st=None, ws_bytes=None,
         **ptrs):
    names = ("q", "k", "v", "o", "do", "lse", "dq", "dk", "dv", "ws")
    p = {n: A + i * MB for i, n in enumerate(names)}
    p.update(ptrs)
    q, k = strides(Hq, Lq, D), strides(Hk, Lk, D)
    need = fa.fa_window_bwd_workspace_bytes(B, Hq, Hk, Lq, Lk, D, window, sinks)
    return fa.fa_window_bwd(*(p[n] for n in names), need if ws_bytes is None else ws_bytes,
                            st or [q, k, k, q, q, q, k, k], B, Hq, Hk, Lq, Lk, D, window, sinks, scale, dtype,
                            None)


SIZES = [
    (dict(dtype=2), BAD),
    (dict(B=-1), BAD),
    (dict(Hq=-1), BAD),
    (dict(Hk=-1), BAD),
    (dict(Hk=0), BAD),
    (dict(Hq=3), BAD),
    (dict(Lq=-1), BAD),
    (dict(Lk=-1), BAD),
    (dict(D=0), BAD),
    (dict(D=96), UNS),
    (dict(window=0), BAD),
    (dict(window=-5), BAD),
    (dict(sinks=-1), BAD),
    (dict(scale=math.nan), BAD),
    (dict(scale=math.inf), BAD),
    (dict(Lk=0), UNS),
    (dict(Lk=1 << 30), UNS),
    (dict(B=1 << 12, Hq=1 << 12, Hk=1 << 12, Lq=1 << 15, Lk=1 << 15), UNS),
    (dict(B=0), OK),
    (dict(Hq=0), OK),
    (dict(q=0), BAD),
    (dict(k=A + MB + 8), BAD),
]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(Lq=0), OK),
    (dict(lse=0), BAD),
    (dict(o=A), BAD),
    (dict(o=A + 4 * MB), BAD),
    (dict(lse=A + 1024), BAD),
    (dict(st=[(8192, 2048, 60)] * 4), BAD),
    (dict(st=[(8192, 0, 64)] * 4), BAD),
])
def test_forward_is_refused(kw, status):
    assert _fwd(**kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(Lq=0), UNS),
    (dict(Lq=0, Lk=0), OK),
    (dict(ws=0), BAD),
    (dict(ws=A + 9 * MB + 4), BAD),
    (dict(ws_bytes=16), BAD),
    (dict(dq=A), BAD),
    (dict(dk=A + 8 * MB), BAD),             # on dv
    (dict(dv=A + 5 * MB), BAD),             # on lse
    (dict(ws=A + 6 * MB), BAD),             # on dq
    (dict(st=[(8192, 2048, 64)] * 7 + [(8192, 2048, 4)]), BAD),
])
def test_backward_is_refused(kw, status):
    assert _bwd(**kw) == status


def test_workspace_sizes():
    need = fa.fa_window_bwd_workspace_bytes
    assert need(2, 4, 2, 300, 300, 64, 8, 0) == 2 * 2 * 4 * 384 * 4 + 16
    assert need(2, 4, 2, 300, 300, 64, 8, 0) == need(2, 4, 2, 300, 500, 64, 8, 0)
    for bad in ((0, 4, 2, 300, 300, 64, 8, 0), (2, 4, 3, 300, 300, 64, 8, 0), (2, 4, 2, 300, 300, 96, 8, 0),
                (2, 4, 2, 300, 300, 64, 0, 0), (2, 4, 2, 300, 0, 64, 8, 0), (2, 4, 2, 300, 300, 64, 8, -1)):
        assert need(*bad) == 0
    # The parts of the first tokens' gradients stay below the documented limit, whatever the sizes.
    most = 0
    for B in (1, 2, 7, 64):
        for Hk in (1, 4, 8):
            for G in (1, 8):
                for L in (1024, 8192, 65536):
                    for window in (1, 128, 1000, 4096):
                        for sinks in (1, 130, 1000, L):
                            rows = 2 * B * Hk * G * L * 4 + 16
                            most = max(most, need(B, Hk * G, Hk, L, L, 128, window, sinks) - rows)
    assert 0 < most <= 65 << 20


def _decode(B=2, Hq=4, Hk=2, D=64, num_pages=16, max_pages=4, window=8, sinks=1, scale=0.125, dtype=0, q8=1,
            ws_bytes=None, **ptrs):
    names = ("q", "kc", "vc", "ke", "ve", "bt", "sl", "o", "lse", "ws")
    p = {n: A + i * 16 * MB for i, n in enumerate(names)}
    p.update(ptrs)
    need = fa.fa_decode_window_workspace_bytes(B, Hq, Hk, D, max_pages, window, sinks)
    return fa.fa_decode_window(*(p[n] for n in names), need if ws_bytes is None else ws_bytes, B, Hq, Hk, D,
                               num_pages, max_pages, window, sinks, scale, dtype, q8, None)


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), BAD),
    (dict(window=-1), BAD),
    (dict(sinks=-1), BAD),
    (dict(dtype=2), BAD),
    (dict(q8=2), BAD),
    (dict(Hq=3), BAD),
    (dict(D=80), UNS),
    (dict(scale=math.nan), BAD),
    (dict(q=0), BAD),
    (dict(ke=0), BAD),
    (dict(o=A), BAD),
    (dict(ws=0), BAD),
    (dict(ws_bytes=16), BAD),
    (dict(ws=A + 16 * MB), BAD),
    (dict(B=0), OK),
])
def test_decode_is_refused(kw, status):
    assert _decode(**kw) == status


def test_decode_workspace():
    need = fa.fa_decode_window_workspace_bytes
    assert need(4, 8, 2, 64, 4096, 1 << 20, 0) == fa.fa_decode_workspace_bytes_ex(4, 8, 2, 64, 4096)
    assert 0 < need(4, 8, 2, 64, 1 << 20, 64, 4) <= fa.fa_decode_workspace_bytes_ex(4, 8, 2, 64, 1 << 20)
    assert need(4, 8, 2, 64, 1 << 20, (1 << 31) - 1, (1 << 31) - 1) == \
        fa.fa_decode_workspace_bytes_ex(4, 8, 2, 64, 1 << 20)
    assert need(4, 8, 2, 64, 16, 0, 0) == need(0, 8, 2, 64, 16, 4, 0) == need(4, 8, 3, 64, 16, 4, 0) == 0


def _chunk(B=2, Hq=4, Hk=2, L=32, D=64, num_pages=16, max_pages=4, window=0, sinks=0, scale=0.125, dtype=0, q8=1,
           ws_bytes=None, st=None, **ptrs):
    names = ("q", "kc", "vc", "ke", "ve", "bt", "sl", "nl", "o", "lse", "ws")
    p = {n: A + i * 64 * MB for i, n in enumerate(names)}
    p.update(ptrs)
    need = fa.fa_attention_paged_workspace_bytes(B, Hq, Hk, L, D, max_pages)
    s = strides(Hq, L, D)
    return fa.fa_attention_paged(*(p[n] for n in names), need if ws_bytes is None else ws_bytes, st or [s, s], B,
                                 Hq, Hk, L, D, num_pages, max_pages, window, sinks, scale, dtype, q8, None)


@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), BAD),
    (dict(sinks=-1), BAD),
    (dict(dtype=2), BAD),
    (dict(q8=2), BAD),
    (dict(B=-1), BAD),
    (dict(L=-1), BAD),
    (dict(Hq=3), BAD),
    (dict(Hk=0), BAD),
    (dict(D=80), UNS),
    (dict(Hq=258), UNS),                    # a group of 129
    (dict(max_pages=1 << 26), UNS),
    (dict(B=1 << 12, L=1 << 24, Hq=2, max_pages=1 << 20), UNS),
    (dict(scale=math.inf), BAD),
    (dict(q=0), BAD),
    (dict(q=A + 8), BAD),
    (dict(o=0), BAD),
    (dict(o=A + 1024), BAD),
    (dict(o=A + 64 * MB), BAD),             # on the keys
    (dict(lse=A), BAD),
    (dict(lse=A + 9 * 64 * MB + 2), BAD),
    (dict(kc=0), BAD),
    (dict(ke=0), BAD),
    (dict(bt=0), BAD),
    (dict(sl=0), BAD),
    (dict(nl=A + 7 * 64 * MB + 2), BAD),
    (dict(o=A + 7 * 64 * MB), BAD),         # on the new lengths
    (dict(ws=0), BAD),
    (dict(ws_bytes=64), BAD),
    (dict(ws=A), BAD),
    (dict(st=[(8192, 2048, 60)] * 2), BAD),
    (dict(B=0), OK),
    (dict(L=0), OK),
    (dict(Hq=0), OK),
])
def test_chunk_is_refused(kw, status):
    assert _chunk(**kw) == status


def test_chunk_workspace():
    need = fa.fa_attention_paged_workspace_bytes
    assert need(64, 64, 8, 4096, 128, 4096) <= 41_000_000
    assert 0 < need(1, 8, 8, 16, 128, 4) < need(64, 64, 8, 4096, 128, 4096)
    # Few rows per cache head, whatever the sizes.
    assert max(need(B, G * Hk, Hk, L, 128, pages) for B in (1, 64, 1024, 4096) for Hk in (1, 8, 128)
               for G in (1, 8, 16) for L in (1, 4, 16) for pages in (1, 64, 4096)) <= 123_000_000
    for bad in ((0, 4, 2, 32, 64, 4), (2, 4, 3, 32, 64, 4), (2, 4, 2, 0, 64, 4), (2, 4, 2, 32, 96, 4)):
        assert need(*bad) == 0
