"""Windows and counts of first tokens that mean nothing are refused alike by every call that takes them, before
anything else of the call is looked at (no GPU work)."""
import pytest
import torch

import tiled_attention_08_gb300 as fa


@pytest.fixture(scope="module", autouse=True)
def binding():
    from tiled_attention_08_gb300 import build
    build.build()


def x(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def calls():
    q, none, kv, row, cache = x(1, 4, 8, 64), x(1, 4, 0, 64), x(1, 2, 8, 64), x(1, 4, 64), x(3, 2, 16, 64)
    same = x(3, 4, 16, 64)  # (as many heads as the queries: another kernel without a window)
    bt, sl, lse = x(1, 3, dtype=torch.int32), x(1, dtype=torch.int32), x(1, 4, 8, dtype=torch.float32)
    return {
        "window_forward": lambda window, sinks: fa.window_forward(q, kv, kv, window, sinks),
        "attention_window": lambda window, sinks: fa.attention_window(q, kv, kv, window, sinks),
        "window_backward": lambda window, sinks: fa.window_backward(q, kv, kv, q, lse, q, window, sinks),
        "without queries": lambda window, sinks: fa.window_backward(none, kv, kv, none, lse[..., :0], none, window,
                                                                    sinks),
        "attention_paged": lambda window, sinks: fa.attention_paged(q, cache, cache, bt, sl, window=window,
                                                                    sinks=sinks),
        "decode_paged": lambda window, sinks: fa.decode_paged(row, cache, cache, bt, sl, window=window, sinks=sinks),
        "equal heads": lambda window, sinks: fa.decode_paged(row, same, same, bt, sl, window=window, sinks=sinks),
    }


CALLS = sorted(calls())
PAGED = ["attention_paged", "decode_paged", "equal heads"]  # window=None: all tokens


@pytest.mark.parametrize("name,window,sinks", [(n, w, s) for n in CALLS for w, s in (
    (0, 0), (-4, 0), (-(1 << 40), 0), (4, -1), (4, -(1 << 40)))] + [(n, None, -1) for n in PAGED])
def test_refused_alike(name, window, sinks):
    with pytest.raises(fa.FaError) as e:
        calls()[name](window, sinks)
    assert isinstance(e.value, fa.FaArgumentError) and isinstance(e.value, ValueError)
    assert e.value.status == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_others_go_on(name):
    """To the next check: these tensors are not on a GPU."""
    for window, sinks in ((1, 0), (1 << 40, 1 << 40), *(((None, 0), (None, 5)) if name in PAGED else ())):
        with pytest.raises(ValueError, match="CUDA tensor"):
            calls()[name](window, sinks)


def test_errors_by_status():
    bad, other = fa.FaError("fa_call", fa.FA_ERR_INVALID_ARG), fa.FaError("fa_call", fa.FA_ERR_UNSUPPORTED)
    assert type(bad) is fa.FaArgumentError and type(other) is fa.FaError
    assert not isinstance(other, ValueError) and isinstance(bad, RuntimeError)
    assert str(bad).startswith("fa_call failed: ") and bad.status == fa.FA_ERR_INVALID_ARG


def test_a_class_derived_from_the_error_stays_itself():
    class Mine(fa.FaError):
        pass

    assert type(Mine("fa_call", fa.FA_ERR_INVALID_ARG)) is Mine
