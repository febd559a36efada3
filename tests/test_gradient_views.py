"""Gradients of outputs and output gradients that are views: o is read where it lies if its heads' elements do, what else is not
packed is copied within the call (no GPU here: the library is a stand-in that looks at what it is handed)."""
import ctypes

import pytest
import torch

from exact_tiled_attention_fattn_gb300 import fattn as F

B, N, Hq, Hkv, d = 2, 5, 4, 2, 64


class Library:
    """Reads o and dout where the real one would (arguments 3 and 5) and keeps their elements."""

    def __init__(self):
        self.got = []
        self.read_in_place = False

    def _call(self, *a, strides=(N * Hq * d, Hq * d, d)):
        read = lambda at, n: torch.frombuffer((ctypes.c_uint8 * (2 * n)).from_address(at), dtype=torch.bfloat16)
        shape = (B, N, Hq)
        full = sum(s * (n - 1) for s, n in zip(strides, shape)) + d
        self.got = [torch.as_strided(read(a[3], full), (*shape, d), (*strides, 1)).flatten().clone(), read(a[5], B * N * Hq * d).clone()]
        self.read_in_place = False
        return F.FATTN_OK

    def fattn_bwd_strided(self, *a):
        self._call(*a, strides=a[23:26])
        self.read_in_place = True
        return F.FATTN_OK

    fattn_bwd = fattn_bwd_shaped = fattn_bwd_sinks = _call
    fattn_bwd_workspace_size = fattn_bwd_shaped_workspace_size = fattn_bwd_sinks_workspace_size = lambda self, *a: 256


def views(x):
    yield x
    yield x.transpose(1, 2).contiguous().transpose(1, 2)                    # heads first in memory
    yield torch.stack([x, x], 3).select(3, 1)                               # every second row of d
    yield torch.cat([x, x], -1)[..., d:]                                    # a slice of a wider projection
    yield torch.cat([x[..., :8], x, x[..., :1]], -1)[..., 8:8 + d]          # rows that are no whole 16 bytes apart
    yield torch.cat([x[..., :4], x, x[..., :4]], -1)[..., 4:4 + d]          # rows that do not begin at 16 bytes
    yield torch.stack([x, x], -1)[..., 0]                                   # elements apart


IN_PLACE = [False, True, True, True, False, False, False]                   # of these views as o


@pytest.mark.parametrize("call", [lambda *a: F.bwd(*a, causal=True), lambda *a: F.bwd_shaped(*a, causal=True),
                                  lambda *a: F.bwd_shaped(*a, window=3, sinks=1)])
def test_views_reach_the_call_packed(monkeypatch, call):
    lib = Library()
    monkeypatch.setattr(F, "load_library", lambda: lib)
    monkeypatch.setattr(F, "_stream_handle", lambda s: 0)
    seen = []
    monkeypatch.setattr(F, "_need_cuda", lambda *t, contiguous=True: seen.append((contiguous, t)))
    z = lambda *s: torch.randn(*s, generator=torch.Generator().manual_seed(sum(s))).to(torch.bfloat16)
    q, k, v, lse = z(B, N, Hq, d), z(B, N, Hkv, d), z(B, N, Hkv, d), torch.zeros(B, Hq, N)
    o, g = z(B, N, Hq, d) + 1, z(B, N, Hq, d) - 1
    for ov, here in zip(views(o), IN_PLACE):
        for gv in views(g):
            seen.clear()
            call(q, k, v, ov, lse, gv)
            assert torch.equal(lib.got[0], o.flatten()) and torch.equal(lib.got[1], g.flatten())
            assert lib.read_in_place == here
            loose = [t for c, ts in seen if not c for t in ts]
            assert any(t is ov for t in loose) and any(t is gv for t in loose)      # their device is looked at
    one = torch.full((1, 1, 1, 1), 2.0, dtype=torch.bfloat16).expand(B, N, Hq, d)   # the gradient of a sum
    call(q, k, v, o, lse, one)
    assert (lib.got[1] == 2).all()
    for bad in (o.transpose(1, 2), o[:1], o[..., :32], o.float()):
        with pytest.raises((ValueError, TypeError)):
            call(q, k, v, bad, lse, g)


def test_abi_refuses_other_strides():
    from exact_tiled_attention_fattn_gb300 import build as fbuild
    fbuild.build()
    lib, A = F.load_library(), 0x100000
    call = lambda o=(1024, 256, 64), shaped=1, cap=0.0, slopes=None, window=3, sinks=1, begin=None, ws=None: lib.fattn_bwd_strided(
        A, A, A, A, A, A, A, A, A, 2, 4, 2, 4, 64, 1, 0.1, shaped, cap, slopes, window, sinks, begin, None, *o, ws, 1 << 30, None)
    assert call() == call(o=(64, 0, 0)) == call(shaped=0, window=0, sinks=0) == F.FATTN_ERR_WORKSPACE       # past the checks
    for bad in ((1024, 256, 4), (1020, 256, 64), (1024, 250, 64), (-1024, 256, 64), (1024, 256, -64)):
        assert call(o=bad) == F.FATTN_ERR_INVALID_ARG
    for bad in (dict(cap=1.0), dict(window=1), dict(sinks=1, window=0), dict(slopes=A, window=0, sinks=0), dict(begin=A, window=0, sinks=0)):
        assert call(shaped=0, **{**dict(window=0, sinks=0), **bad}) == F.FATTN_ERR_INVALID_ARG
    assert call(begin=A) == F.FATTN_ERR_UNSUPPORTED and call(sinks=-1) == F.FATTN_ERR_INVALID_ARG
