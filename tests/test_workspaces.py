"""Workspaces that a call allocates for itself come from the memory of the stream it runs on (without a GPU: the library
and the streams are stand-ins)."""
import contextlib

import pytest
import torch

from exact_tiled_attention_fattn_gb300 import fattn as F


class _Library:
    """Every entry point returns 0, the size functions 1000."""

    def __getattr__(self, name):
        return lambda *a: 1000 if name.endswith("workspace_size") else 0


def _calls():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    q, kc, table = bf(1, 8, 2, 64), bf(4, 16, 2, 64), torch.zeros(1, 4, dtype=torch.int32)
    lse = torch.zeros(1, 2, 8)
    return {
        "bwd": lambda s: F.bwd(q, q, q, q, lse, q, stream=s),
        "decode_paged": lambda s: F.decode_paged(q[0, :1], kc, kc, table, i32(9), 2, stream=s),
        "bwd_shaped": lambda s: F.bwd_shaped(q, q, q, q, lse, q, stream=s),
        "decode_paged_shaped": lambda s: F.decode_paged_shaped(q[0, :1], kc, kc, table, i32(9), 2, stream=s),
        "fwd_paged_shaped": lambda s: F.fwd_paged_shaped(q[0], kc, kc, table, i32(9), i32(0, 8), 8, num_splits=2, stream=s),
    }


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("stream", [None, "other"])
def test_workspace_belongs_to_the_calls_stream(monkeypatch, name, stream):
    current, taken = [None], []
    real = torch.empty

    @contextlib.contextmanager
    def on(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    def empty(*a, **kw):
        if kw.get("dtype") == torch.uint8:
            taken.append(current[0])
        return real(*a, **kw)

    monkeypatch.setattr(F, "load_library", lambda: _Library())
    monkeypatch.setattr(F, "_need_cuda", lambda *a, **kw: None)
    monkeypatch.setattr(F, "_stream_handle", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    _calls()[name](stream)
    assert taken == [stream]
