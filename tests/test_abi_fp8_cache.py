"""The 8-bit paged cache without a GPU: bad arguments are refused on the host before CUDA is touched."""
import pytest
import torch

from exact_tiled_attention_fattn_gb300 import build as fbuild
from exact_tiled_attention_fattn_gb300 import fattn as F

A = 0x100000  # an aligned fake device address: never dereferenced, the calls fail validation first


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return F.load_library()


def _append(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_rope_append_paged_fp8(g("q", A), g("qo", A), g("k", A), g("v", A), g("kc", A), g("vc", A), g("ks", A),
                                           g("vs", A), g("bt", A), g("sl", A), g("cu", A), g("pos", None), g("f", A),
                                           g("B", 2), g("T", 3), g("Hq", 4), g("Hkv", 2), g("d", 64), g("rot", 64),
                                           g("ps", 16), g("maxp", 4), g("np", 8), g("qr", 256), 64, 128, 64, 128, 64, 0,
                                           g("amp", 1.0), None)


def _decode(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_decode_paged_fp8(g("q", A), g("kc", A), g("vc", A), g("ks", A), g("vs", A), g("bt", A), g("sl", A),
                                      g("S", 4), g("o", A), g("lse", A), g("B", 2), g("Hq", 4), g("Hkv", 2), g("d", 64),
                                      g("ps", 16), g("maxp", 4), g("np", 8), g("scale", 0.1), g("cap", 0.0),
                                      g("slopes", None), g("win", 0), g("sinks", 0), g("ws", A), g("wsb", 1 << 30), None)


def _chunk(lib, **kw):
    g = lambda n, x: kw.get(n, x)
    return lib.fattn_fwd_paged_fp8(g("q", A), g("kc", A), g("vc", A), g("ks", A), g("vs", A), g("bt", A), g("sl", A),
                                   g("cu", A), g("o", A), g("lse", A), g("B", 2), g("Hq", 4), g("Hkv", 2), g("d", 64),
                                   g("ps", 16), g("maxp", 4), g("np", 8), g("T", 9), g("mq", 5), 1, g("scale", 0.1),
                                   g("cap", 0.0), g("slopes", None), g("win", 0), g("sinks", 0), g("S", 2), g("ws", A),
                                   g("wsb", 1 << 30), None)


CACHE = [dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(bt=None), dict(sl=None), dict(kc=A + 8),
         dict(vc=A + 4), dict(ks=A + 2), dict(vs=A + 1), dict(bt=A + 2), dict(sl=A + 1), dict(ps=0), dict(maxp=0),
         dict(np=0), dict(Hkv=0), dict(B=-1)]


@pytest.mark.parametrize("bad", CACHE + [dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(cu=None), dict(f=None),
                                         dict(q=A + 1), dict(cu=A + 2), dict(pos=A + 2), dict(rot=63), dict(rot=66),
                                         dict(T=-1), dict(qr=-1), dict(amp=float("nan"))])
def test_append_refuses(lib, bad):
    assert _append(lib, **bad) == F.FATTN_ERR_INVALID_ARG


ATTEND = CACHE + [dict(q=None), dict(o=None), dict(q=A + 8), dict(o=A + 2), dict(lse=A + 2), dict(Hq=3), dict(S=0),
                  dict(scale=float("nan")), dict(cap=-1.0), dict(win=-1), dict(sinks=-1), dict(slopes=A + 1)]


@pytest.mark.parametrize("bad", ATTEND)
def test_decode_refuses(lib, bad):
    assert _decode(lib, **bad) == F.FATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", ATTEND + [dict(cu=None), dict(cu=A + 1), dict(T=-1), dict(mq=-1)])
def test_chunks_refuse(lib, bad):
    assert _chunk(lib, **bad) == F.FATTN_ERR_INVALID_ARG


def test_limits_empty_and_workspaces(lib):
    for call in (_append, _decode, _chunk):
        assert call(lib, d=96, rot=64) == F.FATTN_ERR_UNSUPPORTED
        assert call(lib, ps=20) == F.FATTN_ERR_UNSUPPORTED and call(lib, ps=256) == F.FATTN_ERR_UNSUPPORTED
        assert call(lib, maxp=1 << 28) == F.FATTN_ERR_UNSUPPORTED and call(lib, np=1 << 28) == F.FATTN_ERR_UNSUPPORTED
        assert call(lib, B=0, q=None, k=None, kc=None) == F.FATTN_OK
    assert _append(lib, T=0, k=None) == F.FATTN_OK and _chunk(lib, T=0, q=None) == F.FATTN_OK and _chunk(lib, mq=0) == F.FATTN_OK
    need = lib.fattn_decode_workspace_size(2, 4, 64, 4)
    for ws, n in ((None, need), (A, need - 1), (A + 16, need)):
        assert _decode(lib, ws=ws, wsb=n) == F.FATTN_ERR_WORKSPACE
    size = lib.fattn_fwd_paged_fp8_workspace_size
    need = size(2, 4, 2, 64, 16, 4, 9, 5, 2)
    assert need == 512 + 9 * 4 * 2 * 64 * 4 + 256                               # partials, and the counters
    for ws, n in ((None, need), (A, need - 1), (A + 16, need)):
        assert _chunk(lib, ws=ws, wsb=n) == F.FATTN_ERR_WORKSPACE
    pages = 2 * 4 * 16 * 2 * 64 * 2                                             # a bf16 copy of K or V
    assert size(2, 4, 2, 64, 16, 4, 300, 200, 1) == 2 * pages + 256
    assert size(2, 4, 2, 64, 16, 4, 300, 200, 3) == 2 * pages + 256 + lib.fattn_fwd_paged_shaped_workspace_size(300, 4, 64, 3)
    assert size(0, 4, 2, 64, 16, 4, 9, 5, 2) == size(2, 3, 2, 64, 16, 4, 9, 5, 2) == size(2, 4, 2, 64, 16, 4, 9, 5, 0) == 0


def test_splits():
    for case, S in (((1, 8, 8, 128, 16, 1, 32768), 77), ((4, 32, 8, 128, 64, 6, 12032), 21), ((64, 32, 8, 128, 16, 8, 9000), 3),
                    ((1, 8, 8, 128, 16, 1, 200), 4), ((1, 1, 1, 64, 16, 1, 1), 1), ((0, 8, 8, 64, 16, 1, 100), 2)):
        assert F.choose_fp8_splits(*case, 152) == S, case
    assert F.choose_fp8_splits(2, 32, 8, 128, 16, 2048, 16384, 152) == 1
    assert F.choose_fp8_splits(1, 32, 8, 128, 16, 256, 32768, 152) == F.choose_chunk_splits(1, 32, 128, 256, 32768, 152) > 1


def test_binding_refuses(monkeypatch):
    monkeypatch.setattr(F, "load_library", lambda: None)
    monkeypatch.setattr(F, "_need_cuda", lambda *a, **kw: None)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    codes, sc, f = z(4, 16, 2, 64, dt=torch.uint8), torch.ones(4, 2), torch.zeros(32, dtype=torch.float64)
    good = dict(q=z(1, 4, 64), kcache=codes, vcache=codes, kscale=sc, vscale=sc, block_table=i(1, 4), seqlens=i(1), num_splits=1)
    for bad in (dict(q=z(1, 4, 64).float()), dict(kcache=z(4, 16, 2, 64)), dict(vcache=z(4, 16, 2, 64, dt=torch.float8_e4m3fn)),
                dict(seqlens=i(1).long()), dict(kscale=sc.double())):
        with pytest.raises(TypeError):
            F.decode_paged_fp8(**{**good, **bad})
    for bad in (dict(q=z(4, 64)), dict(kscale=torch.ones(4, 1)), dict(vscale=torch.ones(3, 2)), dict(block_table=i(2, 4)),
                dict(seqlens=i(2)), dict(num_splits=1 << 40), dict(out=z(1, 4, 128))):
        with pytest.raises(ValueError):
            F.decode_paged_fp8(**{**good, **bad})
    base = dict(q=z(3, 4, 64), k=z(3, 2, 64), v=z(3, 2, 64), kcache=codes, vcache=codes, kscale=sc, vscale=sc,
                block_table=i(1, 4), seqlens_k=i(1), cu_seqlens_q=i(2), inv_freq=f)
    for bad in (dict(k=z(3, 2, 64).float()), dict(inv_freq=f.float()), dict(kcache=z(4, 16, 2, 64)), dict(positions=i(3).long())):
        with pytest.raises(TypeError):
            F.rope_append_paged_fp8(**{**base, **bad})
    for bad in (dict(k=z(3, 1, 64), v=z(3, 1, 64)), dict(v=z(2, 2, 64)), dict(q=z(2, 4, 64)), dict(positions=i(4)),
                dict(q=None, out=z(3, 4, 64)), dict(seqlens_k=i(2))):
        with pytest.raises(ValueError):
            F.rope_append_paged_fp8(**{**base, **bad})
    chunk = dict(q=z(3, 4, 64), kcache=codes, vcache=codes, kscale=sc, vscale=sc, block_table=i(1, 4), seqlens_k=i(1),
                 cu_seqlens_q=i(2), max_seqlen_q=3, num_splits=1)
    for bad in (dict(q=z(3, 4, 64).float()), dict(cu_seqlens_q=i(2).long())):
        with pytest.raises(TypeError):
            F.fwd_paged_fp8(**{**chunk, **bad})
    for bad in (dict(lse=torch.zeros(4, 4)), dict(slopes=torch.zeros(3)), dict(max_seqlen_q=1 << 40)):
        with pytest.raises(ValueError):
            F.fwd_paged_fp8(**{**chunk, **bad})
