"""Windows with sinks (the first keys stay visible): forward, gradient, chunks over pages, single tokens. Tolerances as
derived in test_gpu_shaped: P and O (dS and the gradients) rounded to bf16, half a step of 2^-8 each; fp32 scores."""
import math

import numpy as np
import pytest
import torch

from tests import visible_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_shaped import H, alibi, check_fwd, f64, make, score_err

pytestmark = pytest.mark.gpu
nan = lambda *s: torch.full(s, float("nan"), device="cuda")
bf_nan = lambda t: nan(*t.shape).to(torch.bfloat16)

# name: B, N, Hq, Hkv, d, causal, cap, slopes, window, sinks
CASES = {
    "one": (1, 1, 1, 1, 64, True, 0.0, False, 1, 1),
    "three": (2, 3, 2, 1, 128, True, 30.0, True, 1, 1),
    "sink1": (1, 700, 4, 2, 128, True, 0.0, False, 100, 1),
    "sink4": (2, 1100, 2, 1, 64, True, 0.0, False, 64, 4),
    "tile": (1, 900, 2, 2, 128, True, 0.0, False, 130, 128),
    "tile_and_one": (1, 1300, 2, 1, 128, True, 0.0, False, 77, 129),
    "two_tiles": (1, 1029, 4, 1, 64, True, 0.0, False, 200, 256),
    "window1": (1, 515, 1, 1, 128, True, 0.0, False, 1, 3),
    "touching": (1, 640, 2, 2, 64, True, 0.0, False, 128, 130),     # sinks end where a tile's window begins
    "nearly_all": (1, 300, 2, 1, 128, True, 0.0, False, 200, 99),
    "all_sinks": (1, 300, 2, 1, 128, True, 0.0, False, 50, 299),
    "more_than_keys": (1, 200, 1, 1, 64, True, 0.0, False, 20, 2 ** 31 - 1),
    "both_sides": (1, 777, 2, 2, 128, False, 0.0, False, 100, 5),
    "both_sides_tiles": (1, 1000, 4, 2, 64, False, 0.0, False, 30, 300),
    "both_all": (1, 260, 1, 1, 64, False, 0.0, False, 30, 260),
    "cap": (1, 800, 4, 2, 128, True, 20.0, False, 90, 7),
    "cap64": (1, 650, 2, 1, 64, True, 5.0, False, 150, 140),
    "cap_far": (1, 400, 2, 2, 64, True, 300.0, False, 50, 9),
    "cap_both": (1, 520, 2, 1, 128, False, 30.0, False, 64, 20),
    "bias": (1, 700, 8, 2, 128, True, 0.0, True, 100, 6),
    "bias_both": (1, 600, 4, 4, 64, False, 0.0, True, 128, 33),
    "everything": (2, 650, 8, 2, 128, True, 30.0, True, 90, 135),
    "many": (52, 300, 4, 2, 64, True, 0.0, False, 40, 2),            # a group's heads share an item of the dK/dV pass
    "many128": (30, 390, 6, 2, 128, True, 0.0, False, 60, 130),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_gradient(name):
    fa = need_gpu()
    B, N, Hq, Hkv, d, causal, cap, sl, window, sinks = CASES[name]
    q, k, v, do = make(len(name) * 17 + N, B, N, Hq, Hkv, d, 2.0 if cap else 1.0)
    slopes, scale = alibi(Hq) if sl else None, 1 / math.sqrt(d)
    kw = dict(causal=causal, scale=scale, softcap=cap, slopes=None if slopes is None else slopes.cuda(), window=window, sinks=sinks)
    o, lse = bf_nan(q), nan(B, Hq, N)
    qc, kc, vc, dc = q.cuda(), k.cuda(), v.cuda(), do.cuda()
    fa.fwd_shaped(qc, kc, vc, out=o, lse=lse, **kw)
    assert fa.debug_read_status() == 0
    grads = dict(dq=bf_nan(q), dk=bf_nan(k), dv=bf_nan(v))
    fa.bwd_shaped(qc, kc, vc, o, lse, dc, **kw, **grads)
    assert fa.debug_read_status() == 0
    vis = R.window_with_sinks(N, N, 0, causal, window, sinks)
    s = None if slopes is None else f64(slopes)
    for b in range(B) if B < 10 else (0, B // 2, B - 1):
        x = [f64(t[b]) for t in (q, k, v)]
        ref = R.forward(*x, scale, cap, s, vis)
        check_fwd(o[b], lse[b], (*ref[:3], ref[3] + (cap if cap > 128 else 0)), f"{name} sequence {b}")
        g, a, e = R.backward(*x, f64(o[b]), f64(lse[b]), f64(do[b]), scale, cap, s, vis)
        es = 2 * score_err(ref[3].max() + (cap if cap > 128 else 0))
        for n in grads:
            got = f64(grads[n][b])
            assert np.isfinite(got).all(), n
            tol = H * 1.02 * (a[n] + np.abs(g[n])) + es * e[n] + 1e-30
            assert (np.abs(got - g[n]) <= tol).all(), (name, n, (np.abs(got - g[n]) / tol).max())


def test_gradient_against_differences():
    """Directional derivative of the 64-bit forward; o's rounding (2^-8 |o| in D) adds to the gradient's own bound."""
    fa = need_gpu()
    N, Hq, Hkv, d, scale = 300, 2, 1, 64, 0.2
    q, k, v, do = make(5, 1, N, Hq, Hkv, d, 1.5)
    kw = dict(causal=True, scale=scale, window=40, sinks=5)
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = fa.fwd_shaped(*dev, **kw)
    got = dict(zip(("dq", "dk", "dv"), fa.bwd_shaped(*dev, o, lse, do.cuda(), **kw)))
    vis = R.window_with_sinks(N, N, 0, True, 40, 5)
    x = dict(dq=f64(q[0]), dk=f64(k[0]), dv=f64(v[0]))
    _, a, e = R.backward(*x.values(), f64(o[0]), f64(lse[0]), f64(do[0]), scale, 0.0, None, vis)
    rng = np.random.default_rng(0)
    for n in got:
        dirn = rng.standard_normal(x[n].shape)
        f = lambda h: (R.forward(*[x[m] + (h * dirn if m == n else 0) for m in x], scale, 0.0, None, vis)[0] * f64(do[0])).sum()
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        tol = ((H * 1.02 * (a[n] + np.abs(f64(got[n][0]))) + (2e-4 + H) * e[n]) * np.abs(dirn)).sum()
        err = abs((f64(got[n][0]) * dirn).sum() - num)
        assert err <= tol, (n, err, tol, num)


def test_no_sinks_and_sinks_that_hide_nothing():
    """sinks = 0 is the call without them; without a window, or with one that reaches the sinks everywhere, every key is
    seen, as without a window."""
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(8, 1, 500, 4, 2, 128))
    plain = fa.fwd_shaped(q, k, v, causal=True)
    for kw in (dict(sinks=9), dict(window=400, sinks=100), dict(window=1, sinks=499), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1)):
        got = fa.fwd_shaped(q, k, v, causal=True, **kw)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1]), kw
    near = fa.fwd_shaped(q, k, v, causal=True, window=60)
    again = fa.fwd_shaped(q, k, v, causal=True, window=60, sinks=0)
    assert torch.equal(near[0], again[0])
    g = [fa.bwd_shaped(q, k, v, *near, do, causal=True, window=60, **kw) for kw in ({}, dict(sinks=0))]
    assert all(torch.equal(a, b) for a, b in zip(*g))


def pages(g, lens, P, Hkv, d, spare=2):
    per = [-(-n // P) for n in lens]
    perm = torch.randperm(sum(per) + spare, generator=g)
    table, used = torch.full((len(lens), max(per) + 1), -1, dtype=torch.int32), 0
    for b, n in enumerate(per):
        table[b, :n], used = perm[used:used + n].int(), used + n
    kc, vc = (torch.randn(sum(per) + spare, P, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    full = [[c[table[b, :per[b]].long()].reshape(-1, Hkv, d)[:n] for c in (kc, vc)] for b, n in enumerate(lens)]
    return kc, vc, table, full


@pytest.mark.parametrize("P,Hq,Hkv,d,lk,lq,causal,cap,sl,window,sinks", [
    (16, 4, 2, 128, [900, 257, 1, 130], [300, 257, 1, 1], True, 0.0, False, 70, 4),
    (32, 8, 1, 64, [1513, 40, 900], [130, 40, 256], True, 0.0, True, 200, 40),
    (64, 2, 2, 128, [1000, 429], [129, 128], False, 0.0, False, 100, 129),
    (128, 5, 1, 64, [384, 2023], [1, 200], True, 20.0, False, 1, 1),
    (16, 2, 1, 64, [1600, 300], [500, 300], True, 10.0, True, 170, 300)])
def test_paged_chunks(P, Hq, Hkv, d, lk, lq, causal, cap, sl, window, sinks):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq)
    T, pad = sum(lq), 5
    kc, vc, table, full = pages(g, lk, P, Hkv, d)
    q = torch.randn(T + pad, Hq, d, generator=g).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lq)])
    slopes = alibi(Hq) if sl else None
    want = []
    for b in range(len(lk)):
        off = lk[b] - lq[b]
        vis = R.window_with_sinks(lq[b], lk[b], off, causal, window, sinks)
        want.append(R.forward(f64(q[cu[b]:cu[b + 1]]), f64(full[b][0]), f64(full[b][1]), 0.15, cap,
                              None if slopes is None else f64(slopes), vis, off))
        # pages between the sinks' last tile and the first window's first tile are not read: their entries may be anything
        table[b, -(-sinks // 128) * 128 // P:max(off - window + 1, 0) // 128 * 128 // P] = -5
    for S in (1, 3):
        o, lse = bf_nan(q), nan(Hq, T + pad)
        fa.fwd_paged_shaped(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lk, dtype=torch.int32).cuda(),
                            torch.tensor(cu, dtype=torch.int32).cuda(), max(lq), causal=causal, scale=0.15, softcap=cap,
                            slopes=None if slopes is None else slopes.cuda(), window=window, sinks=sinks, out=o, lse=lse,
                            num_splits=S)
        assert fa.debug_read_status() == 0
        for b in range(len(lk)):
            check_fwd(o[cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]], want[b], f"splits {S} sequence {b}")
        assert torch.isnan(o[T:].float()).all() and torch.isnan(lse[:, T:]).all()


@pytest.mark.parametrize("P,Hq,Hkv,d,lens,cap,sl,window,sinks", [
    (16, 8, 2, 128, [1000, 1, 0, 333], 0.0, False, 100, 4),
    (32, 4, 4, 64, [2049, 64, 65], 0.0, True, 65, 33),
    (10, 2, 1, 64, [777, 300], 0.0, True, 50, 14),                  # a gap that ends inside a chunk of 16
    (128, 16, 1, 128, [1500, 129], 20.0, False, 1, 1),
    (16, 20, 1, 64, [900, 40], 0.0, False, 200, 300),
    (64, 5, 5, 128, [640, 639, 641], 0.0, False, 128, 64)])
def test_decode(P, Hq, Hkv, d, lens, cap, sl, window, sinks):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq)
    kc, vc, table, full = pages(g, lens, P, Hkv, d)
    q = torch.randn(len(lens), Hq, d, generator=g).to(torch.bfloat16)
    slopes = alibi(Hq) if sl else None
    want = []
    for b, n in enumerate(lens):
        vis = R.window_with_sinks(1, n, n - 1, True, window, sinks)
        want.append(R.forward(f64(q[b:b + 1]), f64(full[b][0]), f64(full[b][1]), 0.15, cap,
                              None if slopes is None else f64(slopes), vis, n - 1))
        table[b, -(-sinks // P):max(n - window, 0) // P] = -5       # what neither touches is not read
    for S in (1, 2, 7):
        o, lse = bf_nan(q), nan(len(lens), Hq)
        fa.decode_paged_shaped(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), S,
                               scale=0.15, softcap=cap, slopes=None if slopes is None else slopes.cuda(), window=window,
                               sinks=sinks, out=o, lse=lse)
        assert fa.debug_read_status() == 0
        for b in range(len(lens)):
            check_fwd(o[b:b + 1], lse[b][:, None], want[b], f"splits {S} sequence {b}")


def test_gradient_again_and_in_a_graph():
    """The sinks' tiles are worked on in pieces that are added in a fixed order: the same bits on every run, in a captured
    graph as well, with a workspace full of anything."""
    fa = need_gpu()
    for Hkv, N in ((2, 3000), (8, 1500)):                  # (per query head, and a group's heads together)
        q, k, v, do = (t.cuda() for t in make(N, 4, N, 8, Hkv, 128))
        kw = dict(causal=True, window=200, sinks=5)
        o, lse = fa.fwd_shaped(q, k, v, **kw)
        want = fa.bwd_shaped(q, k, v, o, lse, do, **kw)
        ws = torch.full((fa.bwd_sinks_workspace_size(4, 8, Hkv, N, 128, True, 200, 5),), 255, dtype=torch.uint8, device="cuda")
        grads = [torch.empty_like(t) for t in want]
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            fa.bwd_shaped(q, k, v, o, lse, do, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws, **kw)
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert fa.debug_read_status() == 0
            assert all(torch.equal(a, b) for a, b in zip(want, grads))
            ws.fill_(127)


def test_long_sequences_at_their_edges():
    """Rows and keys at the edges of what the sinks and the window make visible, in a sequence of many tiles."""
    fa = need_gpu()
    N, W, S = 6000, 700, 130
    q, k, v, do = make(2, 1, N, 2, 1, 64)
    kw = dict(causal=True, scale=0.125, window=W, sinks=S)
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = fa.fwd_shaped(*dev, **kw)
    g = dict(zip(("dq", "dk", "dv"), fa.bwd_shaped(*dev, o, lse, do.cuda(), **kw)))
    assert fa.debug_read_status() == 0
    vis = R.window_with_sinks(N, N, 0, True, W, S)
    x = [f64(t[0]) for t in (q, k, v)]
    ref = R.forward(*x, 0.125, 0.0, None, vis)
    check_fwd(o[0], lse[0], ref)
    want, a, e = R.backward(*x, f64(o[0]), f64(lse[0]), f64(do[0]), 0.125, 0.0, None, vis)
    es = 2 * score_err(ref[3].max())
    for n in g:
        tol = H * 1.02 * (a[n] + np.abs(want[n])) + es * e[n] + 1e-30
        assert (np.abs(f64(g[n][0]) - want[n]) <= tol).all(), n
