"""Shaped attention (tanh cap, distance bias, window, key ranges): forward, gradient, chunks over pages.

Tolerances. Forward: P is rounded to bf16 (half a step, 2^-8 of it, as l sums the unrounded P) and so is O:
2^-8 (sum p |v| + |O|). fp32: a score is off by at most 1e-6 of the magnitude M behind it plus 5e-5 (128
products summed in fp32; the cap's 1 - 2r, log2 units), and so is lse; P is off by twice that, relatively.
Gradients, from the same o and lse: P and dS rounded to bf16, the result as well: 2^-8 (sum of magnitudes + |g|);
fp32 errors as above on P, dP and D.
"""
import math

import numpy as np
import pytest
import torch

from tests import shaped_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
H = 2.0 ** -8  # half a step of bf16
f64 = lambda t: t.detach().cpu().double().numpy()


def score_err(M):
    return 5e-5 + 1e-6 * M


def check_fwd(o, lse, ref, what=""):
    O, L, A, M = ref
    g, gl = f64(o), f64(lse)
    assert np.isfinite(g).all(), what
    dead = ~np.isfinite(L)
    assert np.array_equal(np.isneginf(gl), dead), what
    assert (np.abs(gl - L)[~dead] <= score_err(M)[~dead] + 2.0 ** -23 * np.abs(L[~dead])).all(), \
        (what, np.abs(gl - L)[~dead].max())
    tol = H * (A + np.abs(O)) * 1.01 + 2 * score_err(M).T[:, :, None] * A
    assert (np.abs(g - O) <= tol).all(), (what, np.abs(g - O).max(), (np.abs(g - O) / np.maximum(tol, 1e-30)).max())


def make(seed, B, N, Hq, Hkv, d, std=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, s=1.0: (torch.randn(B, N, h, d, generator=g) * s).to(torch.bfloat16)
    return r(Hq, std), r(Hkv, std), r(Hkv), r(Hq)


def alibi(Hq):
    return (2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float()


def docs(fa, lens, N, prefix=None, B=1):
    ids = torch.full((B, N), -1, dtype=torch.int64)
    o = 0
    for i, n in enumerate(lens):
        ids[:, o:o + n], o = i, o + n
    return fa.document_ranges(ids, prefix)


# name: B, N, Hq, Hkv, d, causal, cap, slopes, window, documents, prefix
CASES = {
    "one": (1, 1, 1, 1, 64, True, 30.0, True, 1, None, None),
    "three": (2, 3, 2, 1, 128, True, 0.0, True, 2, None, None),
    "plain": (1, 200, 2, 2, 128, False, 0.0, False, 0, None, None),
    "cap128": (2, 300, 4, 2, 128, True, 20.0, False, 0, None, None),
    "cap64": (1, 513, 4, 1, 64, True, 5.0, False, 0, None, None),
    "cap_full": (1, 257, 2, 2, 128, False, 50.0, False, 0, None, None),
    "bias": (1, 700, 8, 2, 128, True, 0.0, True, 0, None, None),
    "bias_both": (1, 385, 4, 4, 64, False, 0.0, True, 0, None, None),
    "window": (1, 900, 2, 1, 128, True, 0.0, False, 100, None, None),
    "window_both": (1, 640, 2, 2, 64, False, 0.0, False, 130, None, None),
    "window1": (1, 129, 1, 1, 128, True, 0.0, False, 1, None, None),
    "window_huge": (1, 300, 1, 1, 64, False, 0.0, False, 2 ** 31 - 1, None, None),
    "docs": (2, 777, 2, 1, 128, True, 0.0, False, 0, [1, 130, 2, 255, 389], None),
    "docs64": (1, 1000, 2, 2, 64, True, 0.0, False, 0, [300, 700], None),
    "docs_both": (1, 600, 2, 2, 128, False, 0.0, False, 0, [128, 128, 1, 300, 43], None),
    "padded": (2, 700, 2, 1, 128, True, 0.0, False, 0, [100, 33], None),       # most rows see nothing
    "padded64": (1, 515, 1, 1, 64, False, 0.0, False, 0, [5], None),
    "prefix": (1, 500, 4, 2, 64, False, 0.0, False, 0, [200, 300], 77),
    "prefix128": (1, 400, 2, 2, 128, False, 0.0, False, 0, [400], 150),
    "all": (2, 650, 4, 2, 128, True, 30.0, True, 90, [123, 27, 400], None),
    "all64": (1, 650, 8, 1, 64, False, 15.0, True, 200, [300, 250], 40),
    # so many key tiles that a group's heads share an item of the dK/dV pass (the cases above take theirs apart)
    "many": (52, 140, 4, 2, 64, True, 20.0, True, 50, [60, 70], None),
    "many128": (40, 130, 6, 2, 128, True, 0.0, False, 0, None, None),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_gradient(name):
    fa = need_gpu()
    B, N, Hq, Hkv, d, causal, cap, sl, window, dl, prefix = CASES[name]
    q, k, v, do = make(len(name) * 31 + N, B, N, Hq, Hkv, d, 2.0 if cap else 1.0)
    slopes = alibi(Hq) if sl else None
    begin, end = docs(fa, dl, N, prefix, B) if dl else (None, None)
    scale = 1 / math.sqrt(d)
    dev = lambda t: None if t is None else t.cuda()
    kw = dict(causal=causal, scale=scale, softcap=cap, slopes=dev(slopes), window=window, key_begin=dev(begin), key_end=dev(end))
    o = torch.full((B, N, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, N), float("nan"), device="cuda")
    fa.fwd_shaped(dev(q), dev(k), dev(v), out=o, lse=lse, **kw)
    assert fa.debug_read_status() == 0
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    grads = dict(dq=nan(q), dk=nan(k), dv=nan(v))
    fa.bwd_shaped(dev(q), dev(k), dev(v), o, lse, dev(do), **kw, **grads)
    assert fa.debug_read_status() == 0
    for b in range(B):
        lo, hi = R.ranges(N, N, 0, causal, window, None if begin is None else begin[b].numpy(),
                          None if end is None else end[b].numpy())
        s = None if slopes is None else f64(slopes)
        ref = R.forward(f64(q[b]), f64(k[b]), f64(v[b]), scale, cap, s, lo, hi)
        check_fwd(o[b], lse[b], ref, f"{name} sequence {b}")
        g, a, e = R.backward(f64(q[b]), f64(k[b]), f64(v[b]), f64(o[b]), f64(lse[b]), f64(do[b]), scale, cap, s, lo, hi)
        es = 2 * score_err(ref[3].max())
        for n in grads:
            got = f64(grads[n][b])
            assert np.isfinite(got).all(), n
            tol = H * 1.02 * (a[n] + np.abs(g[n])) + es * e[n] + 1e-30
            assert (np.abs(got - g[n]) <= tol).all(), (name, n, (np.abs(got - g[n]) / tol).max())


def test_gradient_against_differences():
    """Directional derivative of the 64-bit forward; the bound adds o's rounding (2^-8 |o| in D) to the gradient's own."""
    fa = need_gpu()
    N, Hq, Hkv, d, cap, scale = 150, 2, 1, 64, 10.0, 0.2
    q, k, v, do = make(5, 1, N, Hq, Hkv, d, 1.5)
    slopes = alibi(Hq)
    begin, end = docs(fa, [90, 60], N)
    kw = dict(causal=True, scale=scale, softcap=cap, slopes=slopes.cuda(), window=70, key_begin=begin.cuda(), key_end=end.cuda())
    o, lse = fa.fwd_shaped(q.cuda(), k.cuda(), v.cuda(), **kw)
    got = dict(zip(("dq", "dk", "dv"), fa.bwd_shaped(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), **kw)))
    lo, hi = R.ranges(N, N, 0, True, 70, begin[0].numpy(), end[0].numpy())
    x = dict(dq=f64(q[0]), dk=f64(k[0]), dv=f64(v[0]))
    _, a, e = R.backward(x["dq"], x["dk"], x["dv"], f64(o[0]), f64(lse[0]), f64(do[0]), scale, cap, f64(slopes), lo, hi)
    rng = np.random.default_rng(0)
    for n in got:
        dirn = rng.standard_normal(x[n].shape)
        f = lambda h: (R.forward(*[x[m] + (h * dirn if m == n else 0) for m in ("dq", "dk", "dv")], scale, cap,
                                 f64(slopes), lo, hi)[0] * f64(do[0])).sum()
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        tol = ((H * 1.02 * (a[n] + np.abs(f64(got[n][0]))) + (2e-4 + H) * e[n]) * np.abs(dirn)).sum()
        err = abs((f64(got[n][0]) * dirn).sum() - num)
        assert err <= tol and tol < 0.2 * np.abs(f64(got[n][0]) * dirn).sum(), (n, err, tol, num)


def test_hidden_keys_do_not_leak():
    """Huge and non-finite keys outside the visible range: of no effect on the scores that count."""
    fa = need_gpu()
    q, k, v, _ = make(9, 1, 400, 2, 2, 128)
    begin, end = docs(fa, [150, 250], 400)
    kw = dict(causal=True, key_begin=begin.cuda(), key_end=end.cuda(), softcap=20.0)
    o, lse = fa.fwd_shaped(q.cuda(), k.cuda(), v.cuda(), **kw)
    for bad in (1e30, float("inf"), float("nan")):
        k2 = k.clone()
        k2[:, :150] = bad
        o2, lse2 = fa.fwd_shaped(q.cuda(), k2.cuda(), v.cuda(), **kw)
        assert torch.equal(o2[:, 150:], o[:, 150:]) and torch.equal(lse2[..., 150:], lse[..., 150:])
    assert fa.debug_read_status() == 0


def test_scales_caps_and_slopes_of_any_sign():
    fa = need_gpu()
    q, k, v, _ = make(11, 1, 260, 2, 1, 128)
    lo, hi = R.ranges(260, 260, 0, True, 0)
    for scale, cap, sl in ((-0.2, 0.0, None), (-0.3, 7.0, None), (0.0, 0.0, None), (0.1, 0.0, [-0.01, 0.3]), (-0.1, 0.0, [0.5, 0.0]),
                           (3.0, 25.0, None), (0.088, 1e4, None)):
        s = None if sl is None else torch.tensor(sl)
        o, lse = fa.fwd_shaped(q.cuda(), k.cuda(), v.cuda(), causal=True, scale=scale, softcap=cap, slopes=None if s is None else s.cuda())
        assert fa.debug_read_status() == 0
        O, L, A, M = R.forward(f64(q[0]), f64(k[0]), f64(v[0]), scale, cap, None if s is None else f64(s), lo, hi)
        # the cap's 1 - 2r is off by 2^-22 of the cap, and the raw product by 1e-6 of itself
        check_fwd(o[0], lse[0], (O, L, A, M + cap), f"scale {scale} cap {cap}")


def test_ranges_that_decrease_are_recorded():
    fa = need_gpu()
    q, k, v, _ = make(3, 1, 512, 1, 1, 64)
    end = torch.full((1, 512), 512, dtype=torch.int32)
    end[0, 127] = 60                       # the tile's last row ends below the others
    fa.fwd_shaped(q.cuda(), k.cuda(), v.cuda(), key_end=end.cuda())
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK


@pytest.mark.parametrize("P,Hq,Hkv,d,lk,lq,causal,cap,sl,window,ranged", [
    (16, 4, 2, 128, [700, 257, 1, 130], [300, 257, 1, 1], True, 20.0, False, 0, False),
    (32, 8, 1, 64, [513, 40, 900], [130, 40, 256], True, 0.0, True, 200, False),
    (64, 2, 2, 128, [1000, 129], [129, 128], False, 0.0, True, 300, False),
    (128, 5, 1, 64, [384, 1023], [1, 200], True, 0.0, False, 1, False),
    (16, 2, 1, 64, [600, 300], [500, 300], True, 10.0, True, 170, True)])
def test_paged_chunks(P, Hq, Hkv, d, lk, lq, causal, cap, sl, window, ranged):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq)
    B, T, pad = len(lk), sum(lq), 5
    per = [-(-n // P) for n in lk]
    pages, maxp = sum(per) + 2, max(per) + 1
    perm, table, used = torch.randperm(pages, generator=g), torch.full((B, maxp), -1, dtype=torch.int32), 0
    kc, vc = (torch.randn(pages, P, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T + pad, Hq, d, generator=g).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lq)])
    slopes = alibi(Hq) if sl else None
    begin = end = None
    if ranged:   # two documents per sequence, cut at half its context
        begin, end = torch.zeros(T + pad, dtype=torch.int32), torch.zeros(T + pad, dtype=torch.int32)
    want = []
    for b in range(B):
        table[b, :per[b]], used = perm[used:used + per[b]].int(), used + per[b]
        full = [c[table[b, :per[b]].long()].reshape(-1, Hkv, d)[:lk[b]] for c in (kc, vc)]
        i = np.arange(lq[b]) + lk[b] - lq[b]
        bb, ee = (np.where(i < lk[b] // 2, 0, lk[b] // 2), np.where(i < lk[b] // 2, lk[b] // 2, lk[b])) if ranged else (None, None)
        if ranged:
            begin[cu[b]:cu[b + 1]], end[cu[b]:cu[b + 1]] = torch.from_numpy(bb), torch.from_numpy(ee)
        lo, hi = R.ranges(lq[b], lk[b], lk[b] - lq[b], causal, window, bb, ee)
        want.append(R.forward(f64(q[cu[b]:cu[b + 1]]), f64(full[0]), f64(full[1]), 0.15, cap,
                              None if slopes is None else f64(slopes), lo, hi, off=lk[b] - lq[b]))
        # pages before the first visible tile of 128 are not read: their entries may be anything
        table[b, :(max(int(lo.min()), 0) // 128) * 128 // P] = -5
    dev = lambda t: None if t is None else t.cuda()
    # S runs of every tile's keys: their join adds a few fp32 roundings (2^-24 each), inside the scores' allowance;
    # S = 16 leaves most runs of the short contexts empty
    for S in (1, None, 3, 16):
        o = torch.full((T + pad, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, T + pad), 3.0, device="cuda")
        fa.fwd_paged_shaped(dev(q), dev(kc), dev(vc), dev(table), torch.tensor(lk, dtype=torch.int32).cuda(),
                            torch.from_numpy(cu).int().cuda(), max(lq), causal=causal, scale=0.15, softcap=cap,
                            slopes=dev(slopes), window=window, key_begin=dev(begin), key_end=dev(end), out=o, lse=lse,
                            num_splits=S)
        assert fa.debug_read_status() == 0
        for b in range(B):
            check_fwd(o[cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]], want[b], f"chunk {b}, {S} runs")
        assert bool((o[T:] == 3).all()) and bool((lse[:, T:] == 3).all())  # rows behind the last chunk


def test_split_chunk_keeps_nan_rows_and_repeats():
    """A NaN query row stays NaN through the join, the others are untouched by it, and a second run (and a replay
    of a captured one, over the previous run's partials) gives the same bits."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(4)
    kc, vc = (torch.randn(40, 64, 2, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(300, 4, 128, generator=g).to(torch.bfloat16).cuda()
    table = torch.randperm(40, generator=g).int().reshape(1, 40).cuda()
    ws = torch.full((fa.fwd_paged_shaped_workspace_size(300, 4, 128, 5),), 255, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(4, 300, device="cuda")
    args = (q, kc, vc, table, torch.tensor([2500], dtype=torch.int32).cuda(), torch.tensor([0, 300], dtype=torch.int32).cuda(), 300)
    run = lambda: fa.fwd_paged_shaped(*args, window=900, softcap=20.0, num_splits=5, workspace=ws, out=o, lse=lse)
    run()
    clean = o.clone(), lse.clone()
    q[17, 1] = float("nan")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    assert bool(o[17, 1].isnan().all()) and bool(lse[1, 17].isnan())
    keep = torch.ones(300, 4, dtype=torch.bool, device="cuda")
    keep[17, 1] = False
    # (a warp rescales its rows together, so others may round elsewhere: P and O by 2^-8 each, in both results)
    assert float((o.float() - clean[0].float())[keep].abs().max()) <= 4 * H * float(vc.float().abs().max())
    assert float((lse - clean[1]).T[keep].abs().max()) <= 4 * H
    q[17, 1] = 0.5
    graph.replay()
    again = o.clone(), lse.clone()
    graph.replay()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1]) and bool(torch.isfinite(o).all())
    assert fa.debug_read_status() == 0


@pytest.mark.parametrize("P,Hq,Hkv,d,lens,S,cap,sl,window", [
    (16, 8, 2, 128, [700, 1, 0, 33], 4, 20.0, False, 0),
    (32, 4, 4, 64, [513, 40, 900], 7, 0.0, True, 200),
    (16, 16, 1, 64, [1500, 20], 3, 0.0, True, 1),
    (64, 20, 1, 128, [1000, 129], 5, 30.0, True, 65),
    (3, 2, 1, 64, [50, 7], 2, 0.0, False, 10),
    (16, 2, 2, 128, [600], 1, 0.0, False, 10 ** 9)])
def test_decode(P, Hq, Hkv, d, lens, S, cap, sl, window):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq + d)
    B = len(lens)
    per = [-(-n // P) for n in lens]
    pages, maxp = sum(per) + 2, max(per) + 1
    perm, table, used = torch.randperm(pages, generator=g), torch.full((B, maxp), -1, dtype=torch.int32), 0
    kc, vc = (torch.randn(pages, P, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = (torch.randn(B, Hq, d, generator=g) * 2).to(torch.bfloat16)
    slopes = alibi(Hq) if sl else None
    want = []
    for b, n in enumerate(lens):
        table[b, :per[b]], used = perm[used:used + per[b]].int(), used + per[b]
        if n:
            full = [c[table[b, :per[b]].long()].reshape(-1, Hkv, d)[:n] for c in (kc, vc)]
            lo, hi = R.ranges(1, n, n - 1, True, window)
            want.append(R.forward(f64(q[b:b + 1]), f64(full[0]), f64(full[1]), 0.1, cap, None if slopes is None else f64(slopes),
                                  lo, hi, off=n - 1))
            table[b, :max(int(lo[0]), 0) // P] = -5   # pages before the window are not read
        else:
            want.append((np.zeros((1, Hq, d)), np.full((Hq, 1), -np.inf), np.zeros((1, Hq, d)), np.zeros((Hq, 1))))
    dev = lambda t: None if t is None else t.cuda()
    o, lse = fa.decode_paged_shaped(dev(q), dev(kc), dev(vc), dev(table), torch.tensor(lens, dtype=torch.int32).cuda(), S, scale=0.1,
                                    softcap=cap, slopes=dev(slopes), window=window)
    assert fa.debug_read_status() == 0
    for b in range(B):
        check_fwd(o[b:b + 1], lse[b][:, None], want[b], f"sequence {b}")


def test_unshaped_calls_agree_with_the_plain_ones():
    """With every shape off the shaped kernels compute what the plain ones do, in the same order."""
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(21, 2, 333, 4, 2, 128))
    o, lse = fa.fwd(q, k, v, causal=True)
    o2, lse2 = fa.fwd_shaped(q, k, v, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for x, y in zip(fa.bwd(q, k, v, o, lse, do, causal=True), fa.bwd_shaped(q, k, v, o, lse, do, causal=True)):
        # S scale and the addition of lse round separately in one of them: P differs by 2^-22 |S|, a bf16 step at most
        assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * x.float().abs().max()


def test_streams_graphs_and_timeouts():
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(31, 1, 600, 2, 1, 128))
    kw = dict(causal=True, softcap=20.0, window=200, slopes=alibi(2).cuda())
    o, lse = fa.fwd_shaped(q, k, v, **kw)
    ref = fa.bwd_shaped(q, k, v, o, lse, do, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    bufs = [torch.zeros_like(t) for t in (o, lse, *ref)]
    ws = torch.empty(fa.bwd_shaped_workspace_size(1, 2, 1, 600, 128), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        fa.fwd_shaped(q, k, v, out=bufs[0], lse=bufs[1], stream=s, **kw)
        fa.bwd_shaped(q, k, v, bufs[0], bufs[1], do, dq=bufs[2], dk=bufs[3], dv=bufs[4], workspace=ws, stream=s, **kw)
    for _ in range(2):
        for b in bufs:
            b.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((o, lse, *ref), bufs))
    # the bounded waits run out as in the plain calls, and the next call is right
    assert fa.debug_read_status() == 0
    fa.debug_set_wait_limit(1_000_000, True)
    try:
        fa.fwd_shaped(q, k, v, **kw)
        st = fa.debug_read_status()
        fa.bwd_shaped(q, k, v, o, lse, do, **kw)
        torch.cuda.synchronize()
    finally:
        fa.debug_set_wait_limit(0, False)
    assert st == fa.FATTN_ERR_TIMEOUT and fa.debug_read_status() == fa.FATTN_ERR_TIMEOUT
    assert torch.equal(fa.fwd_shaped(q, k, v, **kw)[0], o) and fa.debug_read_status() == 0


def test_refusals():
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(1, 1, 40, 4, 2, 64))
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    for bad in (dict(slopes=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(4, device="cuda", dtype=torch.float64)),
                dict(key_begin=z(1, 39)), dict(key_end=z(1, 40).long()), dict(softcap=-1.0), dict(softcap=float("nan")),
                dict(softcap=1e-45), dict(window=-1), dict(scale=float("inf")), dict(slopes=torch.zeros(4))):
        with pytest.raises((ValueError, TypeError, fa.FattnError)):
            fa.fwd_shaped(q, k, v, **bad)
        with pytest.raises((ValueError, TypeError, fa.FattnError)):
            fa.bwd_shaped(q, k, v, q, torch.zeros(1, 4, 40, device="cuda"), do, **bad)
    with pytest.raises(fa.FattnError):
        fa.fwd_shaped(torch.zeros(1, 4, 2, 96, device="cuda", dtype=torch.bfloat16), *(torch.zeros(1, 4, 2, 96, device="cuda", dtype=torch.bfloat16),) * 2)


def test_windows_of_any_size():
    """A window that holds every key is no window, whatever its size, to the bit."""
    fa = need_gpu()
    q, k, v, do = (x.cuda() for x in make(11, 2, 300, 4, 2, 64))
    g = torch.Generator().manual_seed(2)
    kc, vc = (torch.randn(40, 16, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table = torch.randperm(40, generator=g).int().reshape(2, 20).cuda()
    lens, cu = torch.tensor([300, 77], dtype=torch.int32).cuda(), torch.tensor([0, 60, 137], dtype=torch.int32).cuda()
    qc, qd = q[0, :137].contiguous(), q[0, :2].contiguous()
    for causal in (True, False):
        kw = dict(causal=causal, softcap=9.0)
        o, lse = fa.fwd_shaped(q, k, v, **kw)
        calls = [lambda w: fa.fwd_shaped(q, k, v, window=w, **kw), lambda w: fa.bwd_shaped(q, k, v, o, lse, do, window=w, **kw),
                 lambda w: fa.fwd_paged_shaped(qc, kc, vc, table, lens, cu, 77, window=w, num_splits=2, **kw),
                 lambda w: fa.decode_paged_shaped(qd, kc, vc, table, lens, 2, softcap=9.0, window=w)]
        for call in calls:
            plain = call(0)
            for w in (320, 10 ** 9, 2 ** 31 - 1, 2 ** 40):
                assert all(torch.equal(x, y) for x, y in zip(call(w), plain)), w
    assert fa.debug_read_status() == 0


def test_two_streams_at_once():
    """Split chunks and per-head gradients of two streams that run at the same time: each as alone, to the bit."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(8)
    calls = []
    for i in range(2):
        q, k, v, do = (x.cuda() for x in make(40 + i, 1, 700 + 200 * i, 8, 2, 64 + 64 * i))
        kw = dict(causal=True, softcap=15.0 + i)
        o, lse = fa.fwd_shaped(q, k, v, **kw)
        kc, vc = (torch.randn(90, 32, 2, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        qc, table = torch.randn(70, 4, 128, generator=g).to(torch.bfloat16).cuda(), torch.randperm(90, generator=g).int().reshape(1, 90).cuda()
        lens, cu = torch.tensor([2800], dtype=torch.int32).cuda(), torch.tensor([0, 70], dtype=torch.int32).cuda()
        calls.append(lambda s, a=(q, k, v, o, lse, do), kw=kw, c=(qc, kc, vc, table, lens, cu, 70): (
            *fa.bwd_shaped(*a, stream=s, **kw), *fa.fwd_paged_shaped(*c, softcap=9.0, num_splits=6, stream=s)))
    alone = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(c(None))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(alone, got) for x, y in zip(a, b))
    assert fa.debug_read_status() == 0


def test_per_head_gradients_against_one_head_at_a_time():
    """The shares of a group's query heads: dk and dv are the sum of the single heads' (fp32 in between, one rounding)."""
    fa = need_gpu()
    q, k, v, do = (x.cuda() for x in make(44, 1, 500, 6, 2, 128))
    kw = dict(causal=True, window=300, softcap=12.0)
    o, lse = fa.fwd_shaped(q, k, v, **kw)
    dq, dk, dv = fa.bwd_shaped(q, k, v, o, lse, do, **kw)
    sk, sv, mk, mv = (torch.zeros(1, 500, 2, 128, device="cuda") for _ in range(4))
    for h in range(6):
        one = lambda t, j: t[:, :, j:j + 1].contiguous()
        a = fa.bwd_shaped(one(q, h), one(k, h // 3), one(v, h // 3), one(o, h), lse[:, h:h + 1].contiguous(), one(do, h), **kw)
        assert torch.equal(a[0], one(dq, h))
        for t, m, x in ((sk, mk, a[1]), (sv, mv, a[2])):
            t[:, :, h // 3:h // 3 + 1] += x.float()
            m[:, :, h // 3:h // 3 + 1] += x.float().abs()
    # each single head's result and the sum are rounded to bf16: half a step of each
    assert ((dk.float() - sk).abs() <= 1.01 * H * (mk + sk.abs()) + 1e-30).all()
    assert ((dv.float() - sv).abs() <= 1.01 * H * (mv + sv.abs()) + 1e-30).all()


def _decreasing(kind):
    """(begin, end) of 300 rows whose ranges decrease, the rows that lose their keys by it, and whether the forward is concerned."""
    b, e = torch.zeros(300, dtype=torch.int32), torch.full((300,), 300, dtype=torch.int32)
    if kind == "last row":                 # a tile's last row sees nothing: its end is below the others'
        e[127] = 0
    elif kind == "padding":                # padding behind a document with an end of 0
        e[:100], e[100:] = 100, 0
    elif kind == "begin":                  # a tile whose first row begins behind its last row's end
        b[0], e[:128] = 290, 128
    elif kind == "inside":                 # inside the tile's range: the forward is right, the gradient of the keys would not be
        e[100] = 60
    elif kind == "begin inside":
        b[40] = 90
    return b, e, kind not in ("inside", "begin inside")


@pytest.mark.parametrize("kind", ["last row", "padding", "begin", "inside", "begin inside"])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_every_decrease_is_recorded(kind, cap):
    """Rows that would lose keys leave DEVICE_CHECK in the status word: in the forward where their keys are outside
    their tile's, in the gradient always."""
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(6, 1, 300, 2, 1, 64))
    b, e, forward = _decreasing(kind)
    kw = dict(key_begin=b[None].cuda(), key_end=e[None].cuda(), softcap=cap)
    o, lse = fa.fwd_shaped(q, k, v, **kw)
    assert fa.debug_read_status() == (fa.FATTN_ERR_DEVICE_CHECK if forward else 0)
    fa.bwd_shaped(q, k, v, o, lse, do, **kw)
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
    table = torch.arange(19, dtype=torch.int32).view(1, 19).cuda()
    kc, vc = (torch.zeros(19, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([300], [0, 300]))
    for S in (1, 3, 16):
        fa.fwd_paged_shaped(q[0], kc, vc, table, n, cu, 300, causal=False, key_begin=b.cuda(), key_end=e.cuda(), softcap=cap, num_splits=S)
        assert fa.debug_read_status() == (fa.FATTN_ERR_DEVICE_CHECK if forward else 0), S


def test_rows_that_see_nothing_record_nothing():
    """Leading, middle and trailing rows without keys whose ranges do not decrease: whole tiles of them, and empty runs."""
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(7, 1, 700, 2, 1, 64))
    b, e = torch.zeros(700, dtype=torch.int32), torch.zeros(700, dtype=torch.int32)
    b[150:400], e[150:400] = 20, 130                   # rows 0 .. 149 see nothing (begin = end = 0)
    b[400:550], e[400:550] = 130, 130                  # nothing again, at the end of the rows before
    b[550:560], e[550:560] = 140, 300
    b[560:], e[560:] = 300, 300
    kw = dict(key_begin=b[None].cuda(), key_end=e[None].cuda())
    o, lse = fa.fwd_shaped(q, k, v, **kw)
    fa.bwd_shaped(q, k, v, o, lse, do, **kw)
    assert fa.debug_read_status() == 0
    live = (b < e).cuda()
    assert torch.equal(torch.isneginf(lse[0, 0]), ~live) and bool((o[0, ~live] == 0).all())
    table = torch.arange(44, dtype=torch.int32).view(1, 44).cuda()
    kc, vc = (torch.zeros(44, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([700], [0, 700]))
    for S in (1, 5):
        fa.fwd_paged_shaped(q[0], kc, vc, table, n, cu, 700, causal=False, key_begin=b.cuda(), key_end=e.cuda(), num_splits=S)
        assert fa.debug_read_status() == 0


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("causal", [False, True])
def test_ends_far_below_zero_and_begins_far_past_the_keys(cap, causal):
    """Any int32 is a bound: leading rows with the lowest end and trailing ones with the highest begin see nothing."""
    fa = need_gpu()
    q, k, v, do = (t.cuda() for t in make(8, 1, 300, 2, 1, 128))
    b, e = torch.full((300,), 3, dtype=torch.int32), torch.full((300,), 2 ** 31 - 1, dtype=torch.int32)
    e[:40], b[280:] = -2 ** 31, 2 ** 31 - 1
    kw = dict(key_begin=b[None].cuda(), key_end=e[None].cuda(), causal=causal, softcap=cap)
    o, lse = fa.fwd_shaped(q, k, v, **kw)
    grads = fa.bwd_shaped(q, k, v, o, lse, do, **kw)
    near = dict(kw, key_begin=b.clamp(0, 300)[None].cuda(), key_end=e.clamp(0, 300)[None].cuda())
    o2, lse2 = fa.fwd_shaped(q, k, v, **near)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip(grads, fa.bwd_shaped(q, k, v, o2, lse2, do, **near)))
    assert bool((o[0, :40] == 0).all()) and bool((o[0, 280:] == 0).all()) and fa.debug_read_status() == 0


def test_hidden_workspaces_on_another_stream():
    """Calls on a busy stream of their own, with tensors taken and filled on the current one meanwhile: as without them."""
    fa = need_gpu()
    q, k, v, do = (x.cuda() for x in make(50, 1, 900, 8, 2, 128))
    o, lse = fa.fwd_shaped(q, k, v, causal=True)
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(90, 32, 2, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table, lens, cu = torch.randperm(90, generator=g).int().reshape(1, 90).cuda(), *(
        torch.tensor(x, dtype=torch.int32).cuda() for x in ([2800], [0, 70]))
    calls = {fa.bwd_shaped_workspace_size(1, 8, 2, 900, 128): lambda s: fa.bwd_shaped(q, k, v, o, lse, do, causal=True, stream=s),
             fa.bwd_workspace_size(1, 8, 900): lambda s: fa.bwd(q, k, v, o, lse, do, causal=True, stream=s),
             fa.fwd_paged_shaped_workspace_size(70, 8, 128, 6): lambda s: fa.fwd_paged_shaped(q[0, :70], kc, vc, table, lens, cu, 70, num_splits=6, stream=s),
             fa.decode_workspace_size(1, 8, 128, 9): lambda s: fa.decode_paged_shaped(q[0, :1], kc, vc, table, lens, 9, stream=s)}
    s = torch.cuda.Stream()
    for need, call in calls.items():
        alone = call(None)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)          # about 10 ms: the call below starts behind it
        got = call(s)
        for _ in range(4):
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(alone, got))
    assert fa.debug_read_status() == 0
