"""Gradients of outputs and output gradients that are views: copied within the call, on its stream (no GPU here: the library
is a stand-in that looks at what it is handed)."""
import ctypes

import pytest
import torch

from exact_tiled_attention_fattn_gb300 import fattn as F

B, N, Hq, Hkv, d = 2, 5, 4, 2, 64


class Library:
    """Takes o and dout where the real one would (arguments 3 and 5) and keeps their elements."""

    def __init__(self):
        self.got = []

    def _call(self, *a):
        self.got = [torch.frombuffer((ctypes.c_uint8 * (B * N * Hq * d * 2)).from_address(a[i]), dtype=torch.bfloat16).clone() for i in (3, 5)]
        return F.FATTN_OK

    fattn_bwd = fattn_bwd_shaped = fattn_bwd_sinks = _call
    fattn_bwd_workspace_size = fattn_bwd_shaped_workspace_size = fattn_bwd_sinks_workspace_size = lambda self, *a: 256


def views(x):
    yield x
    yield x.transpose(1, 2).contiguous().transpose(1, 2)                    # heads first in memory
    yield torch.stack([x, x], 3).select(3, 1)                               # every second row of d
    yield torch.cat([x, x], -1)[..., :d]                                    # a slice of a wider projection
    yield torch.stack([x, x], -1)[..., 0]                                   # elements apart


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
    for ov in views(o):
        for gv in views(g):
            seen.clear()
            call(q, k, v, ov, lse, gv)
            assert torch.equal(lib.got[0], o.flatten()) and torch.equal(lib.got[1], g.flatten())
            loose = [t for c, ts in seen if not c for t in ts]
            assert any(t is ov for t in loose) and any(t is gv for t in loose)      # their device is looked at
    one = torch.full((1, 1, 1, 1), 2.0, dtype=torch.bfloat16).expand(B, N, Hq, d)   # the gradient of a sum
    call(q, k, v, o, lse, one)
    assert (lib.got[1] == 2).all()
    for bad in (o.transpose(1, 2), o[:1], o[..., :32], o.float()):
        with pytest.raises((ValueError, TypeError)):
            call(q, k, v, bad, lse, g)
