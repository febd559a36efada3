"""Key weights and eviction of the paged cache, and the serving path through all the operators.

Tolerance of a weight: every term e^{s - lse} is off by at most 1e-4 + 2e-6 M of itself (its score and lse, M the
largest magnitude behind a score: the bounds of the shaped tests), the fp32 sum by 2^-24 per addition.
"""
import numpy as np
import pytest
import torch

from tests import shaped_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
f64 = lambda t: t.detach().cpu().double().numpy()
i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def pool(seed, lens, P, Hkv, d, spare=2, fill=-1):
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // P) for n in lens]
    perm = torch.randperm(sum(per) + spare, generator=g)
    table, used = torch.full((len(lens), max(per) + 1), fill, dtype=torch.int32), 0
    for b, n in enumerate(per):
        table[b, :n], used = perm[used:used + n].int(), used + n
    kc, vc = (torch.randn(sum(per) + spare, P, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    return kc, vc, table, perm[used:], g


def rows(cache, table, b, n):
    P = cache.shape[1]
    t = np.arange(n)
    return cache[table[b, t // P].long(), torch.from_numpy(t % P)]


def weights_ref(q, k, lse, scale, cap, slopes, lo, hi, off):
    """Sum over queries and the heads of each group of exp(s - lse) [Hkv, L] and the largest magnitude."""
    N, Hq, _ = q.shape
    L, Hkv = k.shape[:2]
    out, mag = np.zeros((Hkv, L)), 0.0
    j = np.arange(L)
    vis = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
    for h in range(Hq):
        s, _, m = R.scores(q[:, h], k[:, h * Hkv // Hq], scale, cap, None if slopes is None else slopes[h], off)
        live = vis & np.isfinite(lse[h])[:, None]
        out[h * Hkv // Hq] += np.where(live, np.exp(np.where(live, s - lse[h][:, None], 0)), 0).sum(0)
        mag = max(mag, m[vis].max(initial=0))
    return out, mag


@pytest.mark.parametrize("P,Hq,Hkv,d,lk,lq,causal,cap,sl,window", [
    (16, 4, 2, 128, [700, 257, 1, 130], [300, 257, 1, 1], True, 0.0, False, 0),
    (32, 8, 1, 64, [513, 40, 900], [1, 1, 1], True, 20.0, True, 200),
    (64, 2, 2, 128, [1000, 129], [129, 128], False, 0.0, True, 300),
    (128, 5, 1, 64, [384, 1023], [1, 200], True, 0.0, False, 1),
    (3, 20, 1, 64, [50, 7, 300], [3, 0, 33], True, 0.0, False, 40),
    (16, 16, 2, 128, [400, 0], [400, 0], True, 30.0, True, 0),
    (32, 6, 2, 64, [2100, 700], [900, 650], True, 0.0, False, 0),      # many steps a tile, rows of 126
    (64, 7, 1, 128, [333], [40], False, 0.0, True, 0),
    (16, 130, 1, 64, [90], [60], True, 0.0, False, 0),                 # a group of more than 128 heads
    (128, 128, 1, 64, [300], [3], True, 0.0, False, 0)])               # one query a step
def test_key_weights(P, Hq, Hkv, d, lk, lq, causal, cap, sl, window):
    fa = need_gpu()
    kc, vc, table, _, g = pool(P + Hq, lk, P, Hkv, d)
    B, T = len(lk), sum(lq)
    cu = np.concatenate([[0], np.cumsum(lq)])
    q = torch.randn(T + 2, Hq, d, generator=g).to(torch.bfloat16)
    lse = torch.full((Hq, T + 2), 1.0)
    slopes = torch.rand(Hq, generator=g) * 0.2 if sl else None
    w = torch.rand(B, Hkv, table.shape[1] * P, generator=g)
    want, mags, terms = w.double().numpy().copy(), [], []
    for b in range(B):
        if lk[b] == 0:
            mags.append(0), terms.append(0)
            continue
        k = f64(rows(kc, table, b, lk[b]))
        lo, hi = R.ranges(lq[b], lk[b], lk[b] - lq[b], causal, window)
        qb = f64(q[cu[b]:cu[b + 1]])
        _, L, _, _ = R.forward(qb, k, k, 0.15, cap, None if slopes is None else f64(slopes), lo, hi, off=lk[b] - lq[b])
        lse[:, cu[b]:cu[b + 1]] = torch.from_numpy(L).float()
        if lq[b] > 2:
            lse[0, cu[b] + 1] = -float("inf")      # a row that is said to have seen nothing
        s, m = weights_ref(qb, k, f64(lse[:, cu[b]:cu[b + 1]]), 0.15, cap, None if slopes is None else f64(slopes), lo, hi, lk[b] - lq[b])
        want[b, :, :lk[b]] = 0.75 * want[b, :, :lk[b]] + s
        mags.append(m), terms.append(lq[b] * (Hq // Hkv))
    table[table < 0] = 10 ** 6                     # entries past a sequence's pages are not read
    kw = dict(causal=causal, scale=0.15, softcap=cap, slopes=None if slopes is None else slopes.cuda(), window=window)
    args = (q.cuda(), kc.cuda(), table.cuda(), i32(lk), i32(cu), max(lq))
    strided = lse.t().contiguous().cuda().t()      # [Hq, T] seen through [T, Hq]: as decoding writes it
    for l in (lse.cuda(), strided):
        wg = w.cuda()
        out = fa.key_weights_paged(*args, l, weights=wg, decay=0.75, out=wg, **kw)
        assert fa.debug_read_status() == 0 and out is wg
        for b in range(B):
            tol = (1.1e-4 + 2e-6 * mags[b] + terms[b] * 2.0 ** -24) * np.abs(want[b]) + 1e-30
            assert (np.abs(f64(out[b]) - want[b]) <= tol).all(), (b, (np.abs(f64(out[b]) - want[b]) / tol).max())
            assert torch.equal(out[b, :, lk[b]:].cpu(), w[b, :, lk[b]:])
    again = fa.key_weights_paged(*args, lse.cuda(), weights=w.cuda(), decay=0.75, **kw)
    assert all(torch.equal(again[b, :, :lk[b]], out[b, :, :lk[b]]) for b in range(B))   # same order of additions
    fresh = fa.key_weights_paged(*args, lse.cuda(), **kw)
    assert all(bool((fresh[b, :, lk[b]:] == 0).all()) for b in range(B))


def test_key_weights_bad_tables_and_lengths():
    fa = need_gpu()
    kc, vc, table, _, _ = pool(1, [100, 60, 30], 16, 1, 64)
    table[0, 2] = 99                                # tokens 32..47 have no page
    q, lse = torch.randn(3, 2, 64).to(torch.bfloat16).cuda(), torch.zeros(2, 3, device="cuda")
    out = torch.full((3, 1, table.shape[1] * 16), -1.0, device="cuda")
    fa.key_weights_paged(q, kc.cuda(), table.cuda(), i32([100, 1000, 30]), i32([0, 1, 2, 3]), 1, lse, out=out)
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
    assert bool((out[0, 0, 32:48] == 0).all()) and bool((out[0, 0, :32] > 0).all()) and bool((out[1] == -1).all())
    assert bool((out[2, 0, :30] > 0).all())


def evict_ref(kc, vc, table, dst, lens, w, keep, recent, first):
    P, Hkv = kc.shape[1], kc.shape[2]
    k2, v2 = kc.clone(), vc.clone()
    B = len(lens)
    cap = dst.shape[1] * P
    wo, kept = torch.zeros(B, Hkv, cap), torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        m = min(n, keep)
        for h in range(Hkv):
            x = w[b, h].numpy()
            mid = range(first, n - recent) if m < n else []
            order = sorted(mid, key=lambda t: (not x[t] == x[t], -x[t] if x[t] == x[t] else 0, t))
            ids = sorted(list(range(n)) if m == n else
                         list(range(first)) + list(range(n - recent, n)) + order[:m - first - recent])
            for s, t in enumerate(ids):
                kept[b, h, s], wo[b, h, s] = t, w[b, h, t]
                d, a = (int(dst[b, s // P]), s % P), (int(table[b, t // P]), t % P)
                k2[d[0], d[1], h], v2[d[0], d[1], h] = kc[a[0], a[1], h], vc[a[0], a[1], h]
    return k2, v2, torch.tensor([min(n, keep) for n in lens], dtype=torch.int32), wo, kept


def same(a, b):
    return torch.equal(torch.nan_to_num(a.cpu().float(), nan=-7.0), torch.nan_to_num(b.float(), nan=-7.0))


@pytest.mark.parametrize("P,Hkv,d,lens,keep,recent,first,kind", [
    (16, 2, 64, [100, 37, 1, 0], 37, 10, 4, "random"),
    (16, 3, 128, [3000, 2000], 1025, 0, 0, "random"),
    (32, 1, 80, [700, 650], 300, 300, 0, "random"),
    (5, 2, 8, [64, 33], 20, 3, 17, "random"),
    (64, 1, 64, [1500, 900], 1000, 7, 1, "ties"),
    (16, 1, 64, [2500], 1, 0, 0, "ties"),
    (16, 2, 64, [500, 400], 123, 5, 2, "special"),
    (16, 1, 64, [50, 20], 64, 0, 0, "random"),
    (128, 1, 1024, [300], 150, 0, 0, "random"),
    (16, 2, 8, [40001, 17000, 3], 5000, 100, 4, "random"),     # more than 16384 tokens: four blocks a head
    (32, 1, 8, [33000, 16385, 0], 20000, 0, 0, "ties"),
    (64, 1, 8, [20000], 19999, 300, 0, "special"),
    (16, 2, 8, [17000] + [40] * 19, 1000, 9, 9, "ties")])       # and with more heads one block
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(P, Hkv, d, lens, keep, recent, first, kind, in_place):
    fa = need_gpu()
    need = [-(-min(n, keep) // P) for n in lens]
    kc, vc, table, spare, g = pool(P + keep, lens, P, Hkv, d, spare=sum(need) + 1)
    w = torch.randn(len(lens), Hkv, table.shape[1] * P, generator=g)
    if kind == "ties":
        w = torch.randint(-1, 2, w.shape, generator=g).float() * torch.where(torch.rand(w.shape, generator=g) < 0.5, 1.0, -0.0)
    if kind == "special":
        pick = torch.randint(0, 5, w.shape, generator=g)
        w = torch.where(pick == 0, float("inf"), torch.where(pick == 1, -float("inf"), torch.where(pick == 2, float("nan"), w)))
    dst = torch.zeros(len(lens), max(need), dtype=torch.int32)
    o = 0
    for b, m in enumerate(need):
        dst[b, :m], o = spare[o:o + m].int(), o + m
    ref = evict_ref(kc, vc, table, table if in_place else dst, lens, w, keep, recent, first)
    kcg, vcg, wg = kc.cuda(), vc.cuda(), w.cuda()
    kw = dict(out_weights=wg) if in_place else dict(dst_table=dst.cuda())
    if in_place and table.shape[1] * P < keep:
        pytest.skip("nothing to cut")
    n, wo, kept = fa.evict_paged(kcg, vcg, table.cuda(), i32(lens), wg, keep, recent=recent, first=first, **kw)
    assert fa.debug_read_status() == 0
    for a, b in zip((kcg, vcg, n, wo, kept), ref):
        assert same(a, b)


def test_evict_refusals_and_bad_tables():
    fa = need_gpu()
    kc, vc, table, spare, _ = pool(2, [60, 40], 16, 2, 64, spare=6)
    w = torch.rand(2, 2, table.shape[1] * 16).cuda()
    base = lambda **kw: fa.evict_paged(kc.cuda(), vc.cuda(), table.cuda(), kw.pop("seqlens", i32([60, 40])), kw.pop("w", w),
                                       kw.pop("keep", 20), **kw)
    sl = i32([60, 40])
    for bad in (dict(keep=0), dict(keep=20, recent=15, first=6), dict(recent=-1), dict(w=w[:, :1]), dict(w=w.double()),
                dict(dst_table=i32([[1], [2]])), dict(dst_table=i32([[1, 2]])), dict(kept=i32([[[0]]])), dict(seqlens=sl, out_seqlens=sl),
                dict(dst_table=i32([[1, 2], [3, 4]]), out_weights=w)):
        with pytest.raises((ValueError, TypeError, fa.FattnError)):
            base(**bad)
    # a destination outside the pool: its rows are not moved; a length past the table: an empty sequence
    kcg, vcg = kc.cuda(), vc.cuda()
    n, _, kept = fa.evict_paged(kcg, vcg, table.cuda(), i32([60, 4000]), w, 20, dst_table=i32([[int(spare[0]), 77], [0, 0]]))
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK and n.tolist() == [20, 0]
    src = rows(kc, table, 0, 60)[kept[0, 0, :16].long().cpu(), 0]
    assert torch.equal(kcg[int(spare[0]), :, 0].cpu(), src)


@pytest.mark.parametrize("captured", [False, True])
def test_serving_path(captured):
    """Prompt chunk, its key weights, eviction in place, then two decode steps, each of append, attention and weights:
    the cache and the answers equal a plain 64-bit run of the same steps. Once more as one captured graph on its own stream."""
    fa = need_gpu()
    B, Hq, Hkv, d, P, keep, cap = 2, 4, 2, 64, 16, 40, 20.0
    plen, maxp = [90, 70], 8
    g = torch.Generator().manual_seed(3)
    f = fa.rope_frequencies(d)[0]
    width = (Hq + 2 * Hkv) * d
    xs = [torch.randn(n, width, generator=g).to(torch.bfloat16) for n in (sum(plen), B, B)]
    table = torch.randperm(2 * maxp, generator=g).view(B, maxp).int()
    pos = [torch.cat([torch.arange(n) for n in plen]), torch.tensor(plen), torch.tensor(plen) + 1]
    cus = [[0, 90, 160], [0, 1, 2], [0, 1, 2]]
    split = lambda x: [x[:, a * d:b * d].view(x.shape[0], b - a, d) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
    kw = dict(softcap=cap, scale=0.125)
    dev = [x.cuda() for x in xs]
    tg, fg, pg = table.cuda(), f.cuda(), [p.int().cuda() for p in pos]
    sl = [i32(plen)] + [torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2)]
    cug = [i32(c) for c in cus]
    zero = lambda: (torch.zeros(2 * maxp, P, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(2 * maxp, P, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(B, Hkv, maxp * P, device="cuda"))
    kc, vc, w = zero()
    kept = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
    after = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.decode_workspace_size(B, Hq, d, 2), dtype=torch.uint8, device="cuda")
    outs = []

    def steps():
        outs.clear()
        qr = fa.rope_append_paged(*split(dev[0]), kc, vc, tg, sl[0], cug[0], fg, positions=pg[0])
        o, lse = fa.fwd_paged_shaped(qr, kc, vc, tg, sl[0], cug[0], 90, **kw)
        fa.key_weights_paged(qr, kc, tg, sl[0], cug[0], 90, lse, weights=w, out=w, **kw)
        fa.evict_paged(kc, vc, tg, sl[0], w, keep, recent=8, first=2, out_weights=w, out_seqlens=after, kept=kept)
        outs.append(o)
        for i in (1, 2):
            torch.add(after, i, out=sl[i])
            qr = fa.rope_append_paged(*split(dev[i]), kc, vc, tg, sl[i], cug[i], fg, positions=pg[i])
            o, lse = fa.decode_paged_shaped(qr, kc, vc, tg, sl[i], 2, workspace=ws, **kw)
            fa.key_weights_paged(qr, kc, tg, sl[i], cug[i], 1, lse.t(), weights=w, decay=0.9, out=w, **kw)
            outs.append(o)

    if captured:
        steps()                                     # the library's first calls come before a capture
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            steps()
        for t in (kc, vc, w):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
    else:
        steps()
    assert fa.debug_read_status() == 0

    # the same in 64 bits, on bf16 caches as the kernels round them
    def rot(x, p):
        ang = p.double().numpy()[:, None] * f.numpy()
        c, s_ = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = f64(x[..., :d // 2]), f64(x[..., d // 2:])
        return torch.from_numpy(np.concatenate([a * c - b * s_, b * c + a * s_], -1)).to(torch.bfloat16)

    K, V, W = [], [], []
    q, k, v = split(xs[0])
    q, k = rot(q, pos[0]), rot(k, pos[0])
    for b in range(B):
        r = slice(cus[0][b], cus[0][b + 1])
        lo, hi = R.ranges(plen[b], plen[b], 0, True, 0)
        O, L, A, M = R.forward(f64(q[r]), f64(k[r]), f64(v[r]), 0.125, cap, None, lo, hi)
        # q and k may be one bf16 step apart from the kernel's where 64 bits round the other way: 2^-7 of a score's terms at most
        assert np.abs(f64(outs[0][r]) - O).max() < 0.05
        wt, _ = weights_ref(f64(q[r]), f64(k[r]), L, 0.125, cap, None, lo, hi, 0)
        ids = kept[b].cpu().numpy()
        for h in range(Hkv):
            mid = np.arange(2, plen[b] - 8)
            cut = np.sort(wt[h, mid])[::-1][keep - 10 - 1]
            # kept and dropped tokens are on the right sides of the threshold, up to the weights' own error
            drop = np.setdiff1d(np.arange(plen[b]), ids[h])
            assert (np.diff(ids[h]) > 0).all() and set([0, 1, *range(plen[b] - 8, plen[b])]) <= set(ids[h])
            assert (wt[h, drop] <= cut * 1.03).all() and (wt[h, np.intersect1d(ids[h], mid)] >= cut * 0.97).all()
        K.append(np.stack([f64(k[r])[ids[h], h] for h in range(Hkv)], 1))
        V.append(np.stack([f64(v[r])[ids[h], h] for h in range(Hkv)], 1))
        W.append(np.stack([wt[h, ids[h]] for h in range(Hkv)]))
    for i in (1, 2):
        q, k, v = split(xs[i])
        q, k = rot(q, pos[i]), rot(k, pos[i])
        for b in range(B):
            K[b], V[b] = np.concatenate([K[b], f64(k[b:b + 1])]), np.concatenate([V[b], f64(v[b:b + 1])])
            n = K[b].shape[0]
            lo, hi = R.ranges(1, n, n - 1, True, 0)
            O, L, _, _ = R.forward(f64(q[b:b + 1]), K[b], V[b], 0.125, cap, None, lo, hi, off=n - 1)
            assert np.abs(f64(outs[i][b]) - O[0]).max() < 0.05
            s, _ = weights_ref(f64(q[b:b + 1]), K[b], L, 0.125, cap, None, lo, hi, n - 1)
            W[b] = 0.9 * np.pad(W[b], ((0, 0), (0, 1))) + s
    for b in range(B):
        n = K[b].shape[0]
        assert np.abs(f64(w[b, :, :n]) - W[b]).max() < 0.03 * W[b].max()
        # cache rows: within a bf16 step of 64 bits (k), equal (v)
        assert np.abs(f64(rows(kc.cpu(), table, b, n)) - K[b]).max() <= 2.0 ** -7 * np.abs(K[b]).max()
        assert np.array_equal(f64(rows(vc.cpu(), table, b, n)), V[b])


def test_key_weights_wait_runs_out():
    """The tensor-core kernel's bounded waits, as in the attention kernels; the next call is right."""
    fa = need_gpu()
    kc, _, table, _, g = pool(6, [500], 16, 1, 64)
    q, lse = torch.randn(100, 2, 64, generator=g).to(torch.bfloat16).cuda(), torch.zeros(2, 100, device="cuda")
    args = (q, kc.cuda(), table.cuda(), i32([500]), i32([0, 100]), 100, lse)
    want = fa.key_weights_paged(*args)
    assert fa.debug_read_status() == 0
    out = torch.full_like(want, -1.0)
    fa.debug_set_wait_limit(1_000_000, True)
    try:
        fa.key_weights_paged(*args, out=out)
        st = fa.debug_read_status()
    finally:
        fa.debug_set_wait_limit(0, False)
    assert st == fa.FATTN_ERR_TIMEOUT and bool((out == -1).all())
    assert torch.equal(fa.key_weights_paged(*args), want) and fa.debug_read_status() == 0


def test_key_weights_refusals():
    fa = need_gpu()
    kc, vc, table, _, _ = pool(4, [20], 16, 2, 64)
    q, lse = torch.randn(1, 4, 64).to(torch.bfloat16).cuda(), torch.zeros(4, 1, device="cuda")
    w = torch.zeros(1, 2, table.shape[1] * 16, device="cuda")
    call = lambda **kw: fa.key_weights_paged(kw.pop("q", q), kc.cuda(), table.cuda(), i32([20]), i32([0, 1]), 1, kw.pop("lse", lse), **kw)
    call(weights=w)
    for bad in (dict(q=q.float()), dict(lse=lse.double()), dict(lse=lse.t()), dict(weights=w[:, :1]), dict(out=w.int()),
                dict(decay=float("nan")), dict(softcap=-1.0), dict(window=-2), dict(slopes=torch.zeros(2, device="cuda")),
                dict(lse=lse.cpu())):
        with pytest.raises((ValueError, TypeError, fa.FattnError)):
            call(**bad)


@pytest.mark.parametrize("P,Hq,lq", [(16, 4, 3), (16, 8, 40), (16, 128, 1), (3, 4, 40)])   # streaming, tensor cores, one query a step, mma
def test_key_weights_windows_of_any_size(P, Hq, lq):
    """A window that holds every key is no window, whatever its size, to the bit; and one query too many for
    max_seqlen_q leaves its sequence's weights alone."""
    fa = need_gpu()
    kc, _, table, _, g = pool(5, [300, 90], P, 1, 64, fill=0)
    q = torch.randn(2 * lq, Hq, 64, generator=g).to(torch.bfloat16).cuda()
    lse = torch.full((Hq, 2 * lq), 3.0, device="cuda")
    args = (q, kc.cuda(), table.cuda(), i32([300, 90]), i32([0, lq, 2 * lq]))
    for causal in (True, False):
        plain = fa.key_weights_paged(*args, lq, lse, causal=causal)
        for window in (table.shape[1] * P, 10 ** 9, 2 ** 31 - 1, 2 ** 40):
            assert torch.equal(fa.key_weights_paged(*args, lq, lse, causal=causal, window=window), plain), window
        near = fa.key_weights_paged(*args, lq, lse, causal=causal, window=299)
        # the first sequence's last query alone no longer sees key 0
        assert torch.equal(near[:, :, 1:], plain[:, :, 1:]) and bool((near[0, :, 0] < plain[0, :, 0]).all())
        assert torch.equal(near[1], plain[1])
    assert fa.debug_read_status() == 0
    out = torch.full((2, 1, table.shape[1] * P), -2.0, device="cuda")
    fa.key_weights_paged(q, kc.cuda(), table.cuda(), i32([300, 90]), i32([0, lq + 1, 2 * lq]), lq, lse, out=out)
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
    assert bool((out[0] == -2).all()) and (bool((out[1, :, :90] > 0).all()) if lq > 1 else bool((out[1] == 0).all()))


@pytest.mark.parametrize("P,lq", [(16, 1), (16, 40), (8, 40)])
def test_pages_past_32_bits(P, lq):
    """A cache of more than 2^31 elements: the serving step, weights and eviction on its last pages give what they
    give on the first ones."""
    fa = need_gpu()
    Hq, Hkv, d, n = 8, 8, 128, 150
    pages = 2 ** 31 // (P * Hkv * d) + 2 * (-(-n // P)) + 2
    per = -(-n // P)
    kc, vc = (torch.empty(pages, P, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(6)
    old = [torch.randn(per, P, Hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    q, k, v = (torch.randn(lq, h, d, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    f = fa.rope_frequencies(d)[0].cuda()
    lens, cu, got = i32([n]), i32([0, lq]), []
    assert (pages - per) * P * Hkv * d > 2 ** 31
    for base in (0, pages - per):
        table, dst = (i32([list(range(x, x + per))]) for x in (base, base - per if base else per))
        kc[base:base + per], vc[base:base + per] = old
        qr = fa.rope_append_paged(q, k, v, kc, vc, table, lens, cu, f)
        if lq == 1:
            o, lse = fa.decode_paged_shaped(qr, kc, vc, table, lens, 2, softcap=20.0, window=100)
            lse = lse.t()
        elif P >= 16:
            o, lse = fa.fwd_paged_shaped(qr, kc, vc, table, lens, cu, lq, softcap=20.0, window=100)
        else:
            o, lse = qr, torch.full((Hq, lq), 5.0, device="cuda")
        w = fa.key_weights_paged(qr, kc, table, lens, cu, lq, lse, softcap=20.0, window=100)
        m, w2, kept = fa.evict_paged(kc, vc, table, lens, w, 70, recent=20, first=3, dst_table=dst)
        x = dst[0].long()
        moved = [c[x].reshape(-1, Hkv, d)[:70].clone() for c in (kc, vc)]
        fa.evict_paged(kc, vc, table, lens, w, 70, recent=20, first=3)
        got.append((o, lse.contiguous(), w, m, w2, kept, *moved, *(c[base:base + per].clone() for c in (kc, vc))))
        assert fa.debug_read_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(got[0][8].reshape(-1, Hkv, d)[:70], got[0][6])     # in place as into other pages


@pytest.mark.parametrize("P,Hq,lq", [(16, 4, 2), (16, 16, 2), (16, 8, 40), (3, 4, 40)])   # streaming (8, 32 rows), tensor cores, mma.sync
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_key_weights_of_a_nan_lse_are_nan(P, Hq, lq, cap):
    """A NaN lse reaches every key that its query sees, and no other: -inf alone says that a row saw nothing."""
    fa = need_gpu()
    n = 300
    kc, _, table, _, g = pool(5, [n], P, 1, 64, fill=0)
    q = torch.randn(lq, Hq, 64, generator=g).to(torch.bfloat16).cuda()
    lse = torch.full((Hq, lq), 3.0, device="cuda")
    run = lambda: fa.key_weights_paged(q, kc.cuda(), table.cuda(), i32([n]), i32([0, lq]), lq, lse, softcap=cap)
    clean = run()
    lse[1, 0] = float("nan")                         # query 0 of the chunk, position n - lq
    out = run()
    seen = n - lq + 1
    assert bool(out[0, 0, :seen].isnan().all()) and torch.equal(out[0, 0, seen:], clean[0, 0, seen:])
    lse[1, 0] = -float("inf")
    assert bool(torch.isfinite(run()).all()) and fa.debug_read_status() == 0


def test_key_weights_stream_wait_runs_out():
    """The streaming kernel's bounded waits: its copies in flight are waited for, no weight of a token is written, and
    the next call is right."""
    fa = need_gpu()
    for n, d, Hq in ((500, 64, 2), (5, 128, 16)):
        kc, _, table, _, g = pool(6, [n], 16, 1, d)
        q, lse = torch.randn(1, Hq, d, generator=g).to(torch.bfloat16).cuda(), torch.zeros(Hq, 1, device="cuda")
        args = (q, kc.cuda(), table.cuda(), i32([n]), i32([0, 1]), 1, lse)
        want = fa.key_weights_paged(*args)
        assert fa.debug_read_status() == 0
        out = torch.full_like(want, -1.0)
        fa.debug_set_wait_limit(1_000_000, True)
        try:
            fa.key_weights_paged(*args, out=out)
            st = fa.debug_read_status()
        finally:
            fa.debug_set_wait_limit(0, False)
        assert st == fa.FATTN_ERR_TIMEOUT and bool((out[..., :n] == -1).all())
        assert torch.equal(fa.key_weights_paged(*args), want) and fa.debug_read_status() == 0


def test_evict_of_nearly_2_31_tokens():
    """The longest table: the walk of the moving blocks passes its last row without leaving 32 bits. Every token lies in
    the pool's first page and goes to its second."""
    fa = need_gpu()
    P, pages = 65536, 32767
    n = P * pages                                       # 2^31 - 65536
    kc, vc = (torch.zeros(2, P, 1, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[0], vc[0] = 1.0, 2.0
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    w = torch.ones(1, 1, n, device="cuda")
    m, _, kept = fa.evict_paged(kc, vc, table, i32([n]), w, n, dst_table=table + 1)
    assert fa.debug_read_status() == 0 and m.item() == n and kept[0, 0, -1].item() == n - 1
    assert bool((kc[1] == 1).all()) and bool((vc[1] == 2).all())
