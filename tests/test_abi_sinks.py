"""Windows with sinks without a GPU: bad arguments are refused on the host before CUDA is touched."""
import pytest
import torch

from exact_tiled_attention_fattn_gb300 import build as fbuild
from exact_tiled_attention_fattn_gb300 import fattn as F

A = 0x100000  # an aligned fake device address: never dereferenced, the calls fail validation first


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return F.load_library()


def _calls(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    sc, cap, sl, win, sinks = g("scale", 0.1), g("cap", 0.0), g("sl", None), g("win", 64), g("sinks", 4)
    yield lib.fattn_fwd_sinks(g("q", A), A, A, A, None, g("B", 2), g("Hq", 4), 2, g("N", 300), g("d", 128), 1, sc, cap, sl,
                              win, sinks, None)
    yield lib.fattn_bwd_sinks(g("q", A), A, A, A, A, A, A, A, A, g("B", 2), g("Hq", 4), 2, g("N", 300), g("d", 128), 1, sc,
                              cap, sl, win, sinks, g("ws", A), 1 << 30, None)
    yield lib.fattn_fwd_paged_sinks(g("q", A), A, A, A, A, A, A, None, g("B", 2), g("Hq", 4), 2, g("d", 128), 16, 8, 64, 100,
                                    g("N", 300), 1, sc, cap, sl, win, sinks, 1, None, 0, None)
    if "B" not in kw and "N" not in kw:
        yield lib.fattn_decode_paged_sinks(g("q", A), A, A, A, A, 4, A, None, 2, g("Hq", 4), 2, g("d", 128), 16, 8, 64, sc,
                                           cap, sl, win, sinks, g("ws", A), 1 << 30, None)


@pytest.mark.parametrize("bad", [dict(sinks=-1), dict(win=-1), dict(cap=-1.0), dict(sl=A + 2), dict(scale=float("inf")),
                                 dict(q=None), dict(q=A + 8), dict(Hq=3), dict(N=-1), dict(B=-1)])
def test_refusals(lib, bad):
    assert set(_calls(lib, **bad)) == {F.FATTN_ERR_INVALID_ARG}


def test_limits_empty_and_workspaces(lib):
    assert set(_calls(lib, d=96)) == {F.FATTN_ERR_UNSUPPORTED}
    assert set(_calls(lib, B=0, q=None)) == {F.FATTN_OK}
    assert list(_calls(lib, ws=None))[1] == list(_calls(lib, ws=None))[3] == F.FATTN_ERR_WORKSPACE


def test_gradient_workspace(lib):
    base, size = lib.fattn_bwd_shaped_workspace_size, lib.fattn_bwd_sinks_workspace_size
    args = (1, 32, 8, 8192, 128)
    assert size(*args, 1, 0, 4) == size(*args, 1, 512, 0) == size(*args, 1, 9000, 4) == size(*args, 1, 100, 8100) == base(*args)
    assert size(*args, 1, 512, 4) == base(*args) + 11 * 2 * 128 * 8 * 128 * 4             # 64 query tiles, 6 a piece
    assert size(*args, 0, 512, 8100) == base(*args) + 0                                   # nearly all keys are sinks
    assert size(1, 8, 2, 997, 64, 0, 100, 17) == base(1, 8, 2, 997, 64) + 4 * 2 * 128 * 8 * 64 * 4   # per query head
    need = size(*args, 1, 512, 4)
    call = lambda ws, n: lib.fattn_bwd_sinks(A, A, A, A, A, A, A, A, A, 1, 32, 8, 8192, 128, 1, 0.1, 0.0, None, 512, 4, ws, n, None)
    assert call(A, need - 1) == call(None, need) == call(A + 16, need) == F.FATTN_ERR_WORKSPACE
    assert F.bwd_sinks_workspace_size(*args, True, 512, 4) == need


def test_sinks_exclude_key_ranges_and_fit_32_bits():
    t = torch.zeros(1, 4, dtype=torch.int32)
    assert F._sinks(0, t, t) == 0 and F._sinks(3) == 3 and F._sinks(2 ** 40) == 2 ** 31 - 1
    for kw in (dict(key_begin=t), dict(key_end=t)):
        with pytest.raises(ValueError):
            F._sinks(1, **kw)
    with pytest.raises(ValueError):
        F._sinks(-2 ** 40)
