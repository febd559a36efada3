"""include/fattn_ops.h without a GPU: every declared entry point is exported and bound, and bad
arguments are refused on the host before CUDA is touched."""
import math
import os
import re

import pytest
import torch

from exact_tiled_attention_fattn_gb300 import build as fbuild
from exact_tiled_attention_fattn_gb300 import fattn as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # an aligned fake device address: never dereferenced, the calls fail validation first


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return F.load_library()


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "fattn_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(fattn_\w+)\s*\(", text))
    assert names == set(F.SIGNATURES_OPS)
    for n in names:
        assert hasattr(lib, n)


def _rope(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_rope(g("q", A), g("qo", A), g("k", A), g("ko", A), g("pos", A), g("period", 1), g("f", A),
                          g("rows", 4), g("Hq", 4), g("Hk", 2), g("d", 128), g("rot", 64), g("qr", 512), 128, 512, 128,
                          256, g("kh", 128), 256, 128, 0, 0, g("amp", 1.0), g("dt", F.FATTN_BF16), None)


@pytest.mark.parametrize("bad", [dict(q=None), dict(qo=None), dict(q=A + 1), dict(ko=None), dict(k=None), dict(f=None),
                                 dict(f=A + 4), dict(rot=63), dict(rot=130), dict(rot=-2), dict(rows=-1), dict(Hq=0),
                                 dict(pos=None, period=0), dict(pos=A + 2), dict(amp=float("nan")), dict(dt=9),
                                 dict(qr=-1), dict(kh=-1), dict(d=0), dict(dt=F.FATTN_FP32, q=A + 2)])
def test_rope_refuses(lib, bad):
    assert _rope(lib, **bad) == F.FATTN_ERR_INVALID_ARG


def test_rope_limits_and_empty(lib):
    assert _rope(lib, d=1026) == F.FATTN_ERR_UNSUPPORTED
    assert _rope(lib, Hq=4095) == F.FATTN_ERR_UNSUPPORTED
    assert _rope(lib, rows=0, q=None, qo=None, k=None, ko=None, Hk=0, pos=None, f=None) == F.FATTN_OK


def _append(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_rope_append_paged(g("q", A), g("qo", A), g("k", A), g("v", A), g("kc", A), A, g("bt", A), g("sl", A),
                                       g("cu", A), None, g("f", A), g("B", 2), g("T", 3), g("Hq", 4), g("Hkv", 2), 64,
                                       g("rot", 64), g("ps", 16), g("maxp", 4), g("np", 8), 256, 64, 128, 64, 128, 64, 0,
                                       g("amp", 1.0), None)


@pytest.mark.parametrize("bad", [dict(qo=None), dict(q=None), dict(k=None), dict(v=None), dict(kc=None), dict(bt=None),
                                 dict(sl=None), dict(cu=None), dict(f=None), dict(ps=0), dict(maxp=0), dict(np=0),
                                 dict(B=-1), dict(Hkv=0), dict(rot=66), dict(bt=A + 2), dict(kc=A + 1),
                                 dict(amp=float("inf"))])
def test_append_refuses(lib, bad):
    assert _append(lib, **bad) == F.FATTN_ERR_INVALID_ARG


def test_append_limits_and_empty(lib):
    assert _append(lib, maxp=1 << 28) == F.FATTN_ERR_UNSUPPORTED
    assert _append(lib, T=0, k=None, v=None, kc=None) == F.FATTN_OK
    assert _append(lib, B=0, k=None) == F.FATTN_OK


def test_rope_frequencies():
    f, a = F.rope_frequencies(8)
    assert a == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    g, _ = F.rope_frequencies(8, scaling="linear", factor=4.0)
    assert torch.equal(g, f / 4)
    g, _ = F.rope_frequencies(8, scaling="base", factor=4.0)
    assert g[0] == 1.0 and abs(g[3].item() * 4 / f[3].item() - 1) < 1e-12
    f, _ = F.rope_frequencies(128)
    g, a = F.rope_frequencies(128, scaling="bands", factor=8.0, original_length=4096)
    assert g[0] == f[0] and g[-1] == f[-1] / 8 and abs(a - 1.2079441541679836) < 1e-15
    assert bool(((g <= f) & (g >= f / 8)).all())
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, base=0.0)):
        with pytest.raises(ValueError):
            F.rope_frequencies(**bad)


@pytest.mark.parametrize("base,dim,length,factor", [(10000.0, 128, 4096, 8.0), (10000.0, 128, 131072, 4.0),
                                                    (10000.0, 64, 128, 2.0), (500000.0, 128, 8192, 16.0), (10000.0, 2, 4096, 4.0)])
def test_rope_bands_follow_the_turns(base, dim, length, factor):
    """Pairs that turn more than beta_fast times over the original length keep their frequency, less than beta_slow have it
    divided, and the ramp between is linear in the pair index with both of its ends where the turns put them, outside the
    head as well."""
    f, _ = F.rope_frequencies(dim, base)
    g, _ = F.rope_frequencies(dim, base, scaling="bands", factor=factor, original_length=length)
    turns = f * length / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32])
    assert torch.allclose(g[turns < 1], f[turns < 1] / factor, rtol=1e-14)
    share = (1 - g / f) / (1 - 1 / factor)
    lo, hi = (dim / 2 * math.log(length / (2 * math.pi * t)) / math.log(base) for t in (32, 1))
    want = ((torch.arange(dim // 2) - math.floor(lo)) / (math.ceil(hi) - math.floor(lo))).clamp(0, 1)
    assert torch.allclose(share, want.double(), atol=1e-6)
    if (base, dim, length) == (10000.0, 128, 131072):
        assert abs((g / f)[63].item() - 0.46) < 1e-12 and abs((g / f)[60].item() - 0.55) < 1e-12


SHAPE_BAD = [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=1e-44), dict(win=-1), dict(sl=A + 2), dict(kb=A + 1),
             dict(ke=A + 3), dict(scale=float("nan"))]


def _shape(kw):
    return kw.get("cap", 0.0), kw.get("sl"), kw.get("win", 0), kw.get("kb"), kw.get("ke")


def _calls(lib, kw):
    g = lambda n, x: kw.get(n, x)
    cap, sl, win, kb, ke = _shape(kw)
    sc = g("scale", 0.1)
    yield lib.fattn_fwd_shaped(g("q", A), A, A, A, None, g("B", 2), g("Hq", 4), 2, g("N", 300), g("d", 128), 1, sc, cap,
                               sl, win, kb, ke, None)
    yield lib.fattn_fwd_paged_shaped(g("q", A), A, A, A, A, A, A, None, g("B", 2), g("Hq", 4), 2, g("d", 128), 16, 8, 64,
                                     100, g("N", 300), 1, sc, cap, sl, win, kb, ke, g("S", 1), g("ws", None), g("wsb", 0), None)
    yield lib.fattn_bwd_shaped(g("q", A), A, A, A, A, A, A, A, A, g("B", 2), g("Hq", 4), 2, g("N", 300), g("d", 128), 1,
                               sc, cap, sl, win, kb, ke, A, 1 << 20, None)
    if "kb" not in kw and "ke" not in kw and "N" not in kw and "B" not in kw:
        yield lib.fattn_decode_paged_shaped(g("q", A), A, A, A, A, 4, A, None, 2, g("Hq", 4), 2, g("d", 128), 16, 8, 64,
                                            sc, cap, sl, win, A, 1 << 20, None)


@pytest.mark.parametrize("bad", SHAPE_BAD + [dict(q=None), dict(q=A + 8), dict(Hq=3), dict(Hq=0), dict(N=-1), dict(B=-1)])
def test_shaped_calls_refuse(lib, bad):
    assert set(_calls(lib, bad)) == {F.FATTN_ERR_INVALID_ARG}


def test_shaped_calls_limits_and_empty(lib):
    assert set(_calls(lib, dict(d=96))) == {F.FATTN_ERR_UNSUPPORTED}
    assert set(_calls(lib, dict(B=0, q=None))) == {F.FATTN_OK}
    assert set(_calls(lib, dict(N=0, q=None))) == {F.FATTN_OK}
    size = lib.fattn_bwd_shaped_workspace_size
    need, vectors = size(2, 4, 2, 300, 128), lib.fattn_bwd_workspace_size(2, 4, 300)
    assert need == vectors + 2 * 384 * 8 + 2 * 2 * 300 * 4 * 128 * 4            # few key tiles: shares per query head
    assert size(2, 4, 4, 300, 128) == vectors + 2 * 384 * 8 and size(2, 0, 1, 3, 64) == size(2, 4, 0, 3, 64) == 0
    assert size(64, 4, 2, 300, 128) == lib.fattn_bwd_workspace_size(64, 4, 300) + 64 * 384 * 8
    for ws, n in ((A, need - 1), (None, need), (A + 16, need)):
        assert lib.fattn_bwd_shaped(A, A, A, A, A, A, A, A, A, 2, 4, 2, 300, 128, 1, 0.1, 0.0, None, 0, None, None, ws,
                                    n, None) == F.FATTN_ERR_WORKSPACE
    assert lib.fattn_fwd_shaped(A, A, A, A, None, 1 << 15, 1 << 10, 1, 1 << 15, 64, 1, 0.1, 0.0, None, 0, None, None,
                                None) == F.FATTN_ERR_UNSUPPORTED


def test_chunk_splits(lib):
    paged = lambda **kw: list(_calls(lib, kw))[1]
    need = lib.fattn_fwd_paged_shaped_workspace_size(100, 4, 128, 3)
    assert need == -(-100 * 4 * 3 * 4 // 256) * 256 + 100 * 4 * 3 * 128 * 4
    assert lib.fattn_fwd_paged_shaped_workspace_size(100, 4, 128, 1) == 0
    assert paged(S=0) == F.FATTN_ERR_INVALID_ARG and paged(S=-1) == F.FATTN_ERR_INVALID_ARG
    for ws, size in ((None, need), (A, need - 1), (A + 16, need)):
        assert paged(S=3, ws=ws, wsb=size) == F.FATTN_ERR_WORKSPACE
    for case, S in (((4, 32, 128, 4096, 100000), 1), ((3, 16, 64, 517, 9000), 1), ((1, 8, 128, 16, 32768), 16),
                    ((2, 16, 128, 512, 4096), 2), ((1, 8, 128, 2048, 16384), 2), ((1, 8, 128, 16, 100), 1),
                    ((0, 8, 128, 16, 900), 1), ((1, 1, 64, 1, 1), 1)):
        assert F.choose_chunk_splits(*case, 152) == S, case


def test_document_ranges():
    ids = torch.tensor([[0, 0, 0, 4, 4, -1, -1], [2, 2, 2, 2, 2, 2, 2]])
    b, e = F.document_ranges(ids)
    assert b.tolist() == [[0, 0, 0, 3, 3, 5, 5], [0] * 7] and e.tolist() == [[3, 3, 3, 5, 5, 5, 5], [7] * 7]
    b, e = F.document_ranges(ids, prefix_len=2)
    assert e.tolist() == [[2, 2, 3, 5, 5, 5, 5], [2, 2, 3, 4, 5, 6, 7]]
    assert bool((b[:, 1:] >= b[:, :-1]).all() and (e[:, 1:] >= e[:, :-1]).all())
    with pytest.raises(ValueError):
        F.document_ranges(ids[0])


def _weights(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_key_weights_paged(g("q", A), g("kc", A), g("bt", A), g("sl", A), g("cu", A), g("lse", A), g("lh", 1), 4,
                                       g("wi", None), g("wo", A), g("B", 2), g("Hq", 4), 2, g("d", 64), g("ps", 16),
                                       g("maxp", 4), 8, g("T", 2), 1, 1, g("scale", 0.1), g("cap", 0.0), g("slopes", None),
                                       g("win", 0), g("decay", 1.0), None)


@pytest.mark.parametrize("bad", [dict(q=None), dict(kc=None), dict(bt=None), dict(sl=None), dict(cu=None), dict(lse=None),
                                 dict(wo=None), dict(q=A + 8), dict(wi=A + 2), dict(lh=-1), dict(Hq=3), dict(B=-1),
                                 dict(ps=0), dict(T=-1), dict(decay=float("inf")), dict(cap=-2.0), dict(win=-1),
                                 dict(scale=float("nan")), dict(slopes=A + 2)])
def test_key_weights_refuse(lib, bad):
    assert _weights(lib, **bad) == F.FATTN_ERR_INVALID_ARG


def test_key_weights_limits_and_empty(lib):
    assert _weights(lib, d=96) == F.FATTN_ERR_UNSUPPORTED
    assert _weights(lib, maxp=1 << 28) == F.FATTN_ERR_UNSUPPORTED
    assert _weights(lib, B=70000) == F.FATTN_ERR_UNSUPPORTED
    assert _weights(lib, B=0, q=None, kc=None) == F.FATTN_OK


def _evict(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_evict_paged(g("kc", A), g("vc", A), g("bt", A), g("sl", A), g("wi", A), g("dt", None), g("so", A + 64),
                                 g("wo", A), g("kept", A), g("B", 2), g("Hkv", 2), g("d", 64), g("ps", 16), g("maxp", 4), 8,
                                 g("dmaxp", 4), g("keep", 20), g("recent", 2), g("first", 1), None)


@pytest.mark.parametrize("bad", [dict(kc=None), dict(vc=None), dict(bt=None), dict(sl=None), dict(wi=None), dict(so=None),
                                 dict(wo=None), dict(kept=None), dict(kc=A + 8), dict(so=A), dict(keep=0), dict(recent=-1),
                                 dict(recent=20), dict(first=-1), dict(dmaxp=3), dict(dt=A, dmaxp=1, wo=A + 64),
                                 dict(dt=A, dmaxp=3), dict(B=-1), dict(Hkv=0), dict(ps=0)])
def test_evict_refuses(lib, bad):
    assert _evict(lib, **bad) == F.FATTN_ERR_INVALID_ARG


def test_evict_limits_and_empty(lib):
    assert _evict(lib, d=60) == F.FATTN_ERR_UNSUPPORTED
    assert _evict(lib, B=40000) == F.FATTN_ERR_UNSUPPORTED
    assert _evict(lib, B=0, kc=None) == F.FATTN_OK
