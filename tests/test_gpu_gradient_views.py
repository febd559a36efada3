"""Gradients of outputs and output gradients that are views give the bits of the packed call: on another stream, and in a
graph that is replayed with new values."""
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [None, dict(causal=True, softcap=20.0), dict(causal=True, window=70, sinks=4),
                                dict(causal=False, window=40, sinks=130)])
def test_views(kw):
    fa = need_gpu()
    B, N, Hq, Hkv, d = 2, 300, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v, do = rnd(B, N, Hq, d), rnd(B, N, Hkv, d), rnd(B, N, Hkv, d), rnd(B, N, Hq, d)
    fwd, bwd = (fa.fwd, fa.bwd) if kw is None else (fa.fwd_shaped, fa.bwd_shaped)
    kw = dict(causal=True) if kw is None else kw
    o, lse = fwd(q, k, v, **kw)
    want = bwd(q, k, v, o, lse, do, **kw)
    heads_first = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)
    wide, odd = torch.cat([o, do], -1), torch.cat([o[..., :1], o], -1)[..., 1:]
    for ov, gv in ((heads_first(o), do), (o, heads_first(do)), (wide[..., :d], wide[..., d:]), (odd, do)):
        assert not (ov.is_contiguous() and gv.is_contiguous())
        assert all(torch.equal(a, b) for a, b in zip(want, bwd(q, k, v, ov, lse, gv, **kw)))
    # a row of o for all
    row = o[:1, :1, :1].expand(B, N, Hq, d)
    assert all(torch.equal(a, b) for a, b in zip(bwd(q, k, v, row.contiguous(), lse, do, **kw), bwd(q, k, v, row, lse, do, **kw)))
    one = torch.ones(1, 1, 1, 1, dtype=torch.bfloat16, device="cuda").expand(B, N, Hq, d)
    assert all(torch.equal(a, b) for a, b in zip(bwd(q, k, v, o, lse, one.contiguous(), **kw), bwd(q, k, v, o, lse, one, **kw)))
    # on another stream: the copies are that stream's, and what the current one allocates meanwhile is not theirs
    ov, gv, side = heads_first(o), heads_first(do), torch.cuda.Stream()
    torch.cuda.synchronize()
    there = bwd(q, k, v, ov, lse, gv, stream=side, **kw)
    junk = [torch.full_like(o, float("nan")) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, there)) and len(junk) == 4
    # in a graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = bwd(q, k, v, ov, lse, gv, **kw)
    for s in (1.0, 0.5):
        gv.copy_(do * s)
        for x in got:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, bwd(q, k, v, o, lse, do * s, **kw)))
    assert fa.debug_read_status() == 0
