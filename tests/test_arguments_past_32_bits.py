"""Integer arguments that a C int does not hold are refused (without a GPU: the library is a stand-in that accepts all)."""
import pytest
import torch

from exact_tiled_attention_fattn_gb300 import fattn as F


class _Library:
    def __getattr__(self, name):
        return lambda *a: 1000 if name.endswith("workspace_size") else 0


def _calls():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    q, kc, table, lse = bf(1, 8, 2, 64), bf(4, 16, 2, 64), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 2, 8)
    chunk = (table, i32(9), i32(0, 8))
    paged = lambda m=8, **kw: F.fwd_paged_shaped(q[0], kc, kc, *chunk, m, **kw)
    decode = lambda s=2, **kw: F.decode_paged_shaped(q[0, :1], kc, kc, table, i32(9), s, **kw)
    weights = lambda m=8, **kw: F.key_weights_paged(q[0], kc, *chunk, m, lse[0], **kw)
    evict = lambda keep=4, **kw: F.evict_paged(kc, kc, table, i32(9), torch.zeros(1, 2, 64), keep, **kw)
    ok = {"fwd": lambda **kw: F.fwd_shaped(q, q, q, **kw), "bwd": lambda **kw: F.bwd_shaped(q, q, q, q, lse, q, **kw),
          "paged": paged, "decode": decode, "weights": weights, "evict": evict}
    bad = [(n, dict(window=-2 ** 40)) for n in ("fwd", "bwd", "paged", "decode", "weights")]
    bad += [(n, dict(m=2 ** 32 + 1)) for n in ("paged", "weights")]
    bad += [("paged", dict(num_splits=2 ** 32 + 1)), ("decode", dict(s=2 ** 32 + 1))]
    bad += [("evict", {n: x}) for n in ("keep", "recent", "first") for x in (2 ** 32 + 4, -2 ** 32 + 4)]
    return ok, bad


@pytest.mark.parametrize("i", range(len(_calls()[1])))
def test_refused(monkeypatch, i):
    monkeypatch.setattr(F, "load_library", lambda: _Library())
    monkeypatch.setattr(F, "_need_cuda", lambda *a, **kw: None)
    monkeypatch.setattr(F, "_stream_handle", lambda s: 0)
    monkeypatch.setattr(F, "_num_sms", lambda d: 152)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: real(0) if isinstance(a[0], tuple) and max(a[0], default=0) > 2 ** 31 else real(*a, **kw))
    ok, bad = _calls()
    name, kw = bad[i]
    ok[name]()
    if "window" in kw:
        ok[name](window=2 ** 40)             # a window that holds every key is none, whatever its size
    with pytest.raises(ValueError):
        ok[name](**kw)
