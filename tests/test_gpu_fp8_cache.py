"""The 8-bit paged cache: append (rotate, quantize, put), single tokens and chunks over it.

Tolerances. Append: a new code is off its value by half a step of E4M3, 2^-4 of it or 2^-10 of the scale (subnormals), and
the rotated value by 1e-6 of its pair in fp32; codes of V and re-scaled old codes are exact. Attention over codes:
P in fp16, 2^-11 of it (half a step) or, where it is subnormal, 2^-25 of the largest p vscale times a code of at most 448;
O rounded to bf16, 2^-8 of it; fp32 scores as in test_gpu_shaped. Chunks of many rows go through the bf16 prefill and have its bound.
"""
import math

import numpy as np
import pytest
import torch

from tests import visible_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_shaped import H, alibi, check_fwd, f64, score_err

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32)


def round_e4m3(x):
    """Nearest E4M3 value, ties to even, saturated at 448 (numpy, 64 bits)."""
    a = np.abs(x)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    y = np.round(a / 2.0 ** (e - 3)) * 2.0 ** (e - 3)
    return np.sign(x) * np.minimum(y, 448.0)


def need_scale(a):
    return np.exp2(np.maximum(np.ceil(np.log2(np.maximum(a, 1e-300) / 448.0)), -100.0))


def rotated(x, pos, f, inter, amp):
    """x [T, H, d] turned in 64 bits."""
    y, r = x.copy(), 2 * len(f)
    ang = pos[:, None].astype(np.float64) * f[None]
    c, s = (amp * np.cos(ang))[:, None], (amp * np.sin(ang))[:, None]
    a, b = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def held(codes, scales, pages, n):
    """The first n tokens that the given pages hold, [n, Hkv, d] in 64 bits."""
    x = f64(codes.view(torch.uint8)[pages].view(E4M3).float()) * f64(scales[pages])[:, None, :, None]
    return x.reshape(-1, *codes.shape[2:])[:n]


def pool(g, lens, P, Hkv, d, spare=2, any_scale=False):
    """Codes (never NaN inside a sequence, NaN in the slots past it), scales, table with unused entries -1, and values."""
    per = [-(-n // P) for n in lens]
    pages = sum(per) + spare
    perm = torch.randperm(pages, generator=g)
    table, used = torch.full((len(lens), max(max(per), 1) + 1), -1, dtype=torch.int32), 0
    out = []
    for _ in range(2):
        codes = (torch.randn(pages, P, Hkv, d, generator=g) * 100).clamp(-448, 448).to(E4M3)
        scale = torch.exp2(torch.randint(-9, -5, (pages, Hkv), generator=g).float())
        if any_scale:
            scale = scale * (1 + torch.rand(pages, Hkv, generator=g))
        out += [codes, scale]
    kc, ks, vc, vs = out
    full = []
    for b, n in enumerate(lens):
        table[b, :per[b]], used = perm[used:used + per[b]].int(), used + per[b]
        pg = table[b, :per[b]].long()
        full.append([held(kc, ks, pg, n), held(vc, vs, pg, n)])
        if n % P:
            for c in (kc, vc):
                c.view(torch.uint8)[pg[-1], n % P:] = 0x7f
    return kc, vc, ks, vs, table, full


@pytest.mark.parametrize("P,Hq,Hkv,d,rot,inter,lk,lq,odd,pos,amp", [
    (16, 4, 2, 128, 128, False, [37, 16, 1, 100], [1, 1, 1, 1], False, False, 1.0),      # single tokens
    (16, 8, 8, 128, 64, True, [700, 20, 333], [300, 20, 33], False, True, 1.2),
    (32, 6, 3, 64, 64, False, [100, 5, 64, 31], [37, 0, 64, 1], False, False, 1.0),
    (64, 5, 1, 64, 32, True, [129, 200], [2, 190], True, False, 1.0),                     # rows on odd addresses
    (128, 2, 2, 128, 6, False, [500, 128], [400, 128], False, True, 0.5),                 # pairs that split a lane's elements
    (16, 0, 5, 64, 0, False, [50, 18], [3, 18], False, False, 1.0),                       # no q, nothing turned
    (128, 3, 1, 128, 128, True, [127, 129, 1000], [1, 2, 700], True, False, 1.0)])
def test_append(P, Hq, Hkv, d, rot, inter, lk, lq, odd, pos, amp):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq + rot)
    kc, vc, ks, vs, table, _ = pool(g, lk, P, Hkv, d, any_scale=True)
    T, pad, B = sum(lq), 3, len(lk)
    cu = np.concatenate([[0], np.cumsum(lq)])
    x = torch.randn(T + pad, (Hq + 2 * Hkv) * d + 3, generator=g) * torch.exp2(torch.randint(-6, 7, (T + pad, 1), generator=g).float())
    x = x.to(torch.bfloat16).cuda()
    at = 1 if odd else 0
    flat = x[:, at:at + (Hq + 2 * Hkv) * d]
    if not odd:
        flat = flat.contiguous()
    q, k, v = (flat[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    t = np.concatenate([np.arange(n - m, n) for n, m in zip(lk, lq)] + [np.zeros(pad, int)])
    p = t * 7 + 1000000 if pos else t
    f = 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    out = torch.full((T + pad, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda") if Hq else None
    dev = [z.cuda() for z in (kc, vc, ks, vs)]
    fa.rope_append_paged_fp8(q if Hq else None, k, v, *dev, table.cuda(), i32(lk).cuda(), i32(cu).cuda(),
                             torch.from_numpy(f).cuda(), positions=i32(p).cuda() if pos else None, interleaved=inter,
                             amplitude=amp, out=out)
    assert fa.debug_read_status() == 0
    kr, size = rotated(f64(k), p, f, inter, amp), amp * np.abs(f64(k)).max(-1, keepdims=True)
    if Hq:
        want = rotated(f64(q), p, f, inter, amp)
        err = np.abs(f64(out)[:T] - want[:T])
        assert (err <= 2.0 ** -8 * np.abs(want[:T]) + 4e-6 * amp * np.abs(f64(q)[:T]).max(-1, keepdims=True)).all()
        assert torch.isnan(out[T:].float()).all()
    for new, codes, old, scale, old_scale, turned in ((kr, dev[0], kc, dev[2], ks, True), (f64(v), dev[1], vc, dev[3], vs, False)):
        got, got_scale = f64(codes.cpu().float()), f64(scale)
        expect, expect_scale, fresh_rows = f64(old.float()), f64(old_scale), np.zeros(old.shape[:2], bool)
        for b in range(B):
            t0 = lk[b] - lq[b]
            for pi in range(t0 // P, -(-lk[b] // P)) if lq[b] else ():
                pg, a, e = int(table[b, pi]), max(t0, pi * P), min(lk[b], (pi + 1) * P)
                rows = new[cu[b] + a - t0:cu[b] + e - t0]                       # [n, Hkv, d]
                amax = np.abs(rows).max((0, 2))
                s = need_scale(amax)
                kept = a - pi * P
                near = np.abs(np.log2(amax / 448.0) - np.round(np.log2(amax / 448.0))) < 1e-5   # either scale will do
                if kept:
                    s = np.maximum(s, expect_scale[pg])
                assert ((got_scale[pg] == s) | near).all(), (b, pi)
                s = got_scale[pg]
                if kept:
                    ratio = (np.float32(1) * f64(old_scale)[pg] / s).astype(np.float32).astype(np.float64)
                    grown = np.where(s > f64(old_scale)[pg], ratio, 1.0)
                    expect[pg] = round_e4m3(expect[pg] * grown[:, None])              # (and the slots past the new tokens)
                y = rows / s[:, None]
                have = got[pg, kept:kept + e - a]
                if turned:
                    lim = 2.0 ** -4 * np.abs(y) * 1.001 + 2.0 ** -10 + (4e-6 * size[cu[b] + a - t0:cu[b] + e - t0]) / s[:, None]
                    assert (np.abs(have - y) <= lim).all(), (b, pi)
                else:
                    assert np.array_equal(have, round_e4m3((rows / s[:, None]).astype(np.float32).astype(np.float64)))
                expect[pg, kept:kept + e - a] = have
                expect_scale[pg] = s
        assert np.array_equal(got, expect, equal_nan=True) and np.array_equal(got_scale, expect_scale)


def test_append_zeros_infinities_and_nan():
    fa = need_gpu()
    kc, vc = (torch.zeros(4, 16, 1, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((4, 1), float("nan"), device="cuda") for _ in range(2))
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.full((3, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    v[1, 0, 5], v[1, 0, 6], v[2, 0, 7] = float("inf"), float("nan"), -float("inf")
    f = torch.zeros(0, dtype=torch.float64, device="cuda")
    fa.rope_append_paged_fp8(None, k, v, kc, vc, ks, vs, i32([[2]]).cuda(), i32([3]).cuda(), i32([0, 3]).cuda(), f)
    assert fa.debug_read_status() == 0
    assert ks[2, 0] == 2.0 ** -100 and (kc == 0).all() and vs[2, 0] == 2.0 ** -7 and torch.isnan(ks[[0, 1, 3]]).all()
    got = vc.view(E4M3).float()[2, :3, 0] / 128
    bad = torch.zeros(3, 64, dtype=torch.bool, device="cuda")
    bad[1, 5] = bad[1, 6] = bad[2, 7] = True
    assert torch.isnan(got[bad]).all() and (got[~bad] == 3.0).all()
    # the largest bf16 values keep a finite scale, and the next token finds the page's
    v = torch.full((1, 1, 64), 3.3e38, dtype=torch.bfloat16, device="cuda")
    fa.rope_append_paged_fp8(None, k[:1] + 1, v, kc, vc, ks, vs, i32([[2]]).cuda(), i32([4]).cuda(), i32([0, 1]).cuda(), f)
    x = (vc.view(E4M3).double() * vs.double()[:, None, :, None])[2, 3, 0]      # (256 * 2^120 is no 32-bit number)
    assert torch.isfinite(vs[2, 0]) and ((x - v[0, 0].double()).abs() <= 2.0 ** -4 * v[0, 0].double()).all()
    assert (kc.view(E4M3).float()[2, 3, 0] * ks[2, 0] == 1).all() and (kc[2, :3] == 0).all()


def test_append_skips_bad_rows():
    fa = need_gpu()
    d, P = 64, 16
    for lens, table, cu in (([40], [[0, 9, 1]], [0, 30]), ([70], [[0, 1, 2]], [0, 30]), ([5], [[0, 1, 2]], [0, 9]),
                            ([40, 40], [[0, 1, 2], [3, 4, 5]], [0, 8, 3]), ([40], [[0, 1, 2]], [-4, 5])):
        kc, vc = (torch.full((6, P, 1, d), 7, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.ones(6, 1, device="cuda") for _ in range(2))
        x = torch.ones(30, 1, d, dtype=torch.bfloat16, device="cuda")
        fa.rope_append_paged_fp8(None, x, x, kc, vc, ks, vs, i32(table).cuda(), i32(lens).cuda(), i32(cu).cuda(),
                                 torch.zeros(0, dtype=torch.float64, device="cuda"))
        assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK, (lens, cu)


def check_codes(o, lse, ref, peak, n, what):
    """peak: the largest p vscale of each row [Hq, N]."""
    O, L, A, M = ref
    go, gl = f64(o), f64(lse)
    dead = ~np.isfinite(L)
    assert np.isfinite(go).all() and np.array_equal(np.isneginf(gl), dead), what
    off = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, L))
    assert (off <= score_err(M) + 2.0 ** -22 * np.abs(np.where(dead, 0, L))).all(), (what, off.max())
    tol = H * np.abs(O) * 1.01 + (2.0 ** -11 + 2 * score_err(M).T[:, :, None]) * A + (2.0 ** -25 * 448 * n * peak).T[:, :, None]
    assert (np.abs(go - O) <= tol).all(), (what, np.abs(go - O).max(), (np.abs(go - O) / np.maximum(tol, 1e-30)).max())


def peaks(q, k, vscale, scale, cap, slopes, vis, off, lse):
    """The largest p vscale of each row and head, [Hq, N]; vscale [L, Hkv]."""
    N, Hq, _ = q.shape
    out = np.zeros((Hq, N))
    for h in range(Hq):
        s, _, _ = R.scores(q[:, h], k[:, h * k.shape[1] // Hq], scale, cap, None if slopes is None else slopes[h], off)
        live = np.isfinite(lse[h])
        p = np.where(vis & live[:, None], np.exp(np.where(vis, s, 0) - np.where(live, lse[h], 0)[:, None]), 0)
        out[h] = (p * vscale[:, h * k.shape[1] // Hq][None]).max(1, initial=0)
    return out


@pytest.mark.parametrize("P,Hq,Hkv,d,lens,cap,sl,window,sinks,any_scale", [
    (16, 8, 2, 128, [1000, 1, 0, 333, 15, 16, 17], 0.0, False, 0, 0, False),
    (32, 4, 4, 64, [2049, 64, 65], 0.0, False, 0, 0, True),
    (64, 16, 2, 128, [700, 129], 0.0, False, 0, 0, True),
    (128, 16, 1, 128, [1500, 129], 20.0, False, 0, 0, False),           # 16 rows
    (16, 20, 1, 64, [900, 40], 0.0, True, 0, 0, False),                 # 20 rows, three tiles of 8
    (16, 10, 2, 128, [3000, 41], 30.0, True, 100, 0, False),
    (32, 8, 2, 128, [2500, 300, 64], 0.0, False, 64, 4, False),
    (16, 5, 5, 64, [1900, 640, 641], 0.0, True, 128, 64, True),
    (128, 9, 1, 128, [2000, 1], 0.0, False, 1, 1, False),
    (64, 2, 2, 64, [3001], 5.0, False, 700, 200, False),
    (16, 72, 1, 128, [500, 0, 33], 0.0, False, 0, 0, False),            # groups of 24 rows of one query
    (32, 80, 2, 64, [1200, 31], 25.0, True, 90, 10, True)])
def test_decode(P, Hq, Hkv, d, lens, cap, sl, window, sinks, any_scale):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq)
    kc, vc, ks, vs, table, full = pool(g, lens, P, Hkv, d, any_scale=any_scale)
    q = torch.randn(len(lens), Hq, d, generator=g).to(torch.bfloat16)
    slopes = alibi(Hq) if sl else None
    sn = None if slopes is None else f64(slopes)
    want = []
    for b, n in enumerate(lens):
        vis = R.window_with_sinks(1, n, n - 1, True, window, sinks)
        ref = R.forward(f64(q[b:b + 1]), *full[b], 0.15, cap, sn, vis, n - 1)
        vt = np.repeat(f64(vs[table[b, :-(-n // P)].long()]), P, 0)[:n]
        want.append((ref, peaks(f64(q[b:b + 1]), full[b][0], vt, 0.15, cap, sn, vis, n - 1, ref[1])))
        if window:
            table[b, -(-sinks // P):max(n - window, 0) // P] = -5        # what neither touches is not read
    # (a table with room for long contexts: the sequences' steps shared in one line, else by clusters)
    wide = torch.nn.functional.pad(table, (0, 8000), value=-1)
    for S, table in ((1, table), (2, table), (7, table), (16, table), (2, wide), (7, wide), (200, wide)):
        o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((len(lens), Hq), float("nan"), device="cuda")
        fa.decode_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), i32(lens).cuda(), S, scale=0.15,
                            softcap=cap, slopes=None if slopes is None else slopes.cuda(), window=window, sinks=sinks, out=o,
                            lse=lse)
        assert fa.debug_read_status() == 0
        for b, n in enumerate(lens):
            check_codes(o[b:b + 1], lse[b][:, None], *want[b], n, f"splits {S} sequence {b}")


CHUNKS = [  # P, Hq, Hkv, d, lk, lq, causal, cap, slopes, window, sinks, any scale
    (16, 8, 2, 128, [1000, 257, 5, 18], [6, 6, 5, 1], True, 0.0, False, 0, 0, True),
    (64, 4, 4, 64, [1513, 40, 900], [13, 40, 7], True, 0.0, True, 0, 0, False),
    (32, 16, 2, 128, [700, 130], [20, 17], False, 0.0, False, 0, 0, False),
    (128, 6, 2, 64, [1000, 429], [9, 30], True, 20.0, False, 100, 3, False),
    (16, 4, 2, 128, [2000, 300], [8, 20], False, 0.0, False, 70, 40, True),
    (64, 8, 2, 128, [1200, 129, 60], [6, 5, 6], True, 30.0, False, 0, 0, False),                  # 24 rows
    (16, 8, 1, 64, [800, 90], [4, 3], True, 0.0, True, 150, 20, True),                            # 32 rows
    (32, 12, 2, 64, [500, 77, 1000], [7, 6, 2], False, 0.0, False, 0, 0, False),                  # 42 rows, groups of 24
    (16, 8, 2, 128, [3000, 64], [60, 60], True, 0.0, False, 0, 0, False),                         # 240 rows, the most in groups of 4
    (16, 4, 2, 128, [900, 257, 1, 130], [300, 257, 1, 1], True, 0.0, False, 0, 0, False),         # through the prefill from here
    (32, 8, 1, 64, [1513, 40, 900], [130, 40, 256], True, 0.0, True, 200, 40, False),
    (64, 8, 2, 128, [1000, 429], [129, 128], False, 20.0, False, 100, 129, False),
    (128, 20, 1, 64, [384, 2023], [1, 200], True, 0.0, False, 1, 1, False)]


@pytest.mark.parametrize("P,Hq,Hkv,d,lk,lq,causal,cap,sl,window,sinks,any_scale", CHUNKS)
def test_chunks(P, Hq, Hkv, d, lk, lq, causal, cap, sl, window, sinks, any_scale):
    fa = need_gpu()
    g = torch.Generator().manual_seed(P + Hq + lq[0])
    kc, vc, ks, vs, table, full = pool(g, lk, P, Hkv, d, any_scale=any_scale)
    T, pad = sum(lq), 4
    q = torch.randn(T + pad, Hq, d, generator=g).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lq)])
    slopes = alibi(Hq) if sl else None
    sn = None if slopes is None else f64(slopes)
    streamed = max(lq) * (Hq // Hkv) <= fa.fp8_stream_rows(Hq // Hkv)
    want = []
    for b in range(len(lk)):
        off, x = lk[b] - lq[b], f64(q[cu[b]:cu[b + 1]])
        vis = R.window_with_sinks(lq[b], lk[b], off, causal, window, sinks)
        ref = R.forward(x, *full[b], 0.15, cap, sn, vis, off)
        vt = np.repeat(f64(vs[table[b, :-(-lk[b] // P)].long()]), P, 0)[:lk[b]]
        want.append((ref, peaks(x, full[b][0], vt, 0.15, cap, sn, vis, off, ref[1])))
        if window:
            table[b, -(-sinks // 128) * 128 // P:max(off - window + 1, 0) // 128 * 128 // P] = -5
    wide = [torch.nn.functional.pad(table, (0, 8000), value=-1)] if streamed else []
    for S, table in ((1, table), (3, table), (9, table), *((S, t) for S in (3, 64) for t in wide)):
        o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, T + pad), float("nan"), device="cuda")
        fa.fwd_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), i32(lk).cuda(), i32(cu).cuda(), max(lq),
                         causal=causal, scale=0.15, softcap=cap, slopes=None if slopes is None else slopes.cuda(), window=window,
                         sinks=sinks, out=o, lse=lse, num_splits=S)
        assert fa.debug_read_status() == 0
        for b in range(len(lk)):
            mine = o[cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]]
            if streamed:
                check_codes(*mine, *want[b], lk[b], f"splits {S} sequence {b}")
            else:
                check_fwd(*mine, want[b][0], f"splits {S} sequence {b}")
        assert torch.isnan(o[T:].float()).all() and torch.isnan(lse[:, T:]).all()
    table = table[:, :table.shape[1] - 8000 * len(wide)].contiguous()
    again = fa.fwd_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), i32(lk).cuda(), i32(cu).cuda(),
                             max(lq), causal=causal, scale=0.15, softcap=cap, slopes=None if slopes is None else slopes.cuda(),
                             window=window, sinks=sinks)
    assert (again[0][:T].float() - o[:T].float()).abs().max() <= 2 ** -5 * o[:T].float().abs().max()


def test_uneven_scales_keep_what_weighs():
    """One page of tiny values holds nearly all the weight: the output is as exact as that page's values. And scores of q far
    from 1 in size."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(1)
    kc, vc, ks, vs, table, _ = pool(g, [300], 16, 1, 128)
    vs[:] = 2.0 ** -3
    vs[table[0, 3].long()] = 2.0 ** -40
    q = torch.randn(1, 4, 128, generator=g).to(torch.bfloat16)
    kc.view(torch.uint8)[table[0, 3].long(), 5] = (q[0, 0] * 100).clamp(-448, 448).to(E4M3).view(torch.uint8)
    for size in (1.0, 2.0 ** -60, 2.0 ** 40):
        full = [held(c, s, table[0, :19].long(), 300) for c, s in ((kc, ks), (vc, vs))]
        qs = (q.float() * size).to(torch.bfloat16)
        scale = 0.5 / size
        vis = np.ones((1, 300), bool)
        ref = R.forward(f64(qs), *full, scale, 0.0, None, vis)
        pk = peaks(f64(qs), full[0], np.repeat(f64(vs[table[0, :19].long()]), 16, 0)[:300], scale, 0.0, None, vis, 0, ref[1])
        o, lse = fa.decode_paged_fp8(qs.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), i32([300]).cuda(), 2, scale=scale)
        check_codes(o, lse.t(), ref, pk, 300, size)


def test_bad_pages_and_lengths_are_recorded():
    fa = need_gpu()
    g = torch.Generator().manual_seed(2)
    kc, vc, ks, vs, table, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in pool(g, [100, 100], 16, 2, 64))
    q = torch.randn(2, 4, 64, generator=g).to(torch.bfloat16).cuda()
    for lens, entry in (([100, 100], 99), ([100, 100], -3), ([100, 1000], None), ([-1, 100], None)):
        t = table.clone()
        if entry is not None:
            t[1, 2] = entry
        o, lse = fa.decode_paged_fp8(q, kc, vc, ks, vs, t, i32(lens).cuda(), 3)
        assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
        if entry is not None:
            assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    for cu in ([0, 5, 3], [0, 1, 9], [-1, 1, 2]):
        fa.fwd_paged_fp8(q, kc, vc, ks, vs, table, i32([100, 100]).cuda(), i32(cu).cuda(), 2)
        assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK


def test_serving_steps_together():
    """A prompt in two chunks, then single tokens, with a window and sinks: rotated, quantized, attended; against the 64-bit
    attention over the values that the cache holds, and a graph of the step that is replayed as the sequences grow."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(4)
    P, Hq, Hkv, d, B, W, S = 16, 8, 2, 128, 2, 90, 4
    maxp = 24
    perm = torch.randperm(B * maxp, generator=g).int().view(B, maxp).cuda()
    kc, vc = (torch.full((B * maxp, P, Hkv, d), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(B * maxp, Hkv, device="cuda") for _ in range(2))
    inv_freq, _ = fa.rope_frequencies(d, device="cuda")
    kw = dict(scale=0.1, window=W, sinks=S)

    def check(q, o, lse, lens, lq):
        r = 0
        for b in range(B):
            off = lens[b] - lq[b]
            vis = R.window_with_sinks(lq[b], lens[b], off, True, W, S)
            ref = R.forward(f64(q[r:r + lq[b]]), *(held(c, s, perm[b, :-(-lens[b] // P)].long(), lens[b]) for c, s in ((kc, ks), (vc, vs))), 0.1, 0.0, None, vis, off)
            check_fwd(o[r:r + lq[b]], lse[:, r:r + lq[b]], ref, f"{lens}")
            r += lq[b]

    lens = [0, 0]
    for lq in ([200, 77], [30, 100]):
        lens = [a + b for a, b in zip(lens, lq)]
        T = sum(lq)
        x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
        cu = i32([0, lq[0], T]).cuda()
        q = fa.rope_append_paged_fp8(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, ks, vs, perm, i32(lens).cuda(), cu, inv_freq)
        o, lse = fa.fwd_paged_fp8(q, kc, vc, ks, vs, perm, i32(lens).cuda(), cu, max(lq), **kw)
        assert fa.debug_read_status() == 0
        check(q, o, lse, lens, lq)
    # single tokens from a captured graph
    x = torch.empty(B, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    n, cu = i32(lens).cuda(), i32([0, 1, 2]).cuda()
    qr, o, lse = (torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)), None, torch.empty(B, Hq, device="cuda")
    qr, o = qr
    ws = torch.empty(fa.decode_workspace_size(B, Hq, d, 3), dtype=torch.uint8, device="cuda")

    def step():
        n.add_(1)
        fa.rope_append_paged_fp8(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, ks, vs, perm, n, cu, inv_freq, out=qr)
        fa.decode_paged_fp8(qr, kc, vc, ks, vs, perm, n, 3, out=o, lse=lse, workspace=ws, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(20):
        x.copy_(torch.randn(x.shape, generator=g) * (1 + 3 * (i == 9)))       # token 9 outgrows its page's scales
        graph.replay()
        assert fa.debug_read_status() == 0
        lens = [a + 1 for a in lens]
        assert n.tolist() == lens
        check(qr, o, lse.t(), lens, [1, 1])


def test_pool_past_2_31_bytes():
    """Pages whose first byte lies past 2^31 of both caches, and rows of the bf16 copy's tables with them."""
    fa = need_gpu()
    P, Hq, Hkv, d = 128, 16, 8, 128
    pages = 2 ** 31 // (P * Hkv * d) + 40
    kc, vc = (torch.empty(pages, P, Hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, Hkv, device="cuda") for _ in range(2))
    table = torch.arange(pages - 12, pages, dtype=torch.int32, device="cuda").view(2, 6).flip(1).contiguous()
    g = torch.Generator().manual_seed(6)
    lens = [700, 650]
    T = sum(lens)
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    cu, n = i32([0, 700, T]).cuda(), i32(lens).cuda()
    inv_freq, _ = fa.rope_frequencies(d, device="cuda")
    q = fa.rope_append_paged_fp8(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, ks, vs, table, n, cu, inv_freq)
    o, lse = fa.fwd_paged_fp8(q, kc, vc, ks, vs, table, n, cu, 700, scale=0.1)
    last = torch.stack([q[699], q[T - 1]])
    od, ld = fa.decode_paged_fp8(last, kc, vc, ks, vs, table, n, 3, scale=0.1)
    assert fa.debug_read_status() == 0
    for b, n in enumerate(lens):
        pg = table[b, :-(-n // P)].long()
        full = [held(kc[pg], ks[pg], torch.arange(len(pg)), n), held(vc[pg], vs[pg], torch.arange(len(pg)), n)]
        rows = [0, 1, 127, 300, n - 1]
        vis = np.tril(np.ones((n, n), bool))[rows]
        at = torch.tensor(rows) + (0 if b == 0 else 700)
        ref = R.forward(f64(q[at.cuda()]), *full, 0.1, 0.0, None, vis)
        check_fwd(o[at.cuda()], lse[:, at.cuda()], ref, f"sequence {b}")
        check_fwd(od[b:b + 1], ld[b][:, None], tuple(z[-1:] if z.ndim == 3 else z[:, -1:] for z in ref), f"token of sequence {b}")


def test_same_results_on_another_stream_and_again():
    """A call on another stream than the current one, its workspace its own; and every call gives the same bits again."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(3)
    lens = [3000, 77, 1500]
    kc, vc, ks, vs, table, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in pool(g, lens, 16, 2, 128))
    n = i32(lens).cuda()
    q1 = torch.randn(3, 8, 128, generator=g).to(torch.bfloat16).cuda()
    qs = torch.randn(90, 8, 128, generator=g).to(torch.bfloat16).cuda()
    few, many = i32([0, 5, 9, 15]).cuda(), i32([0, 60, 70, 90]).cuda()
    wide = torch.nn.functional.pad(table, (0, 8000), value=-1)
    side = torch.cuda.Stream()

    def calls(stream):
        return [*fa.decode_paged_fp8(q1, kc, vc, ks, vs, table, n, 5, stream=stream),
                *fa.decode_paged_fp8(q1, kc, vc, ks, vs, wide, n, 50, stream=stream),
                *fa.fwd_paged_fp8(qs[:15], kc, vc, ks, vs, wide, n, few, 6, stream=stream, num_splits=9),
                *fa.fwd_paged_fp8(qs[:15], kc, vc, ks, vs, table, n, few, 6, stream=stream),
                *fa.fwd_paged_fp8(qs, kc, vc, ks, vs, table, n, many, 60, stream=stream, num_splits=2)]

    here = calls(None)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    there = calls(side)
    again = calls(None)                                   # at the same time
    torch.cuda.synchronize()
    assert fa.debug_read_status() == 0
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(here, there, again))


def test_empty_problems_and_graphs_that_share_a_workspace():
    fa = need_gpu()
    g = torch.Generator().manual_seed(8)
    kc, vc, ks, vs, table, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in pool(g, [900, 0], 32, 2, 64))
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
    none = table[:0].contiguous()
    zero = i32([0]).cuda()
    o, lse = fa.decode_paged_fp8(e(0, 4, 64), kc, vc, ks, vs, none, e(0, dt=torch.int32), 2)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    fa.fwd_paged_fp8(e(0, 4, 64), kc, vc, ks, vs, none, e(0, dt=torch.int32), zero, 0)
    fa.rope_append_paged_fp8(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), kc, vc, ks, vs, none, e(0, dt=torch.int32), zero,
                             torch.zeros(32, dtype=torch.float64, device="cuda"))
    # two graphs over one workspace, replayed in turn, each with a row count of its own
    n, cu = i32([900, 0]).cuda(), (i32([0, 1, 1]).cuda(), i32([0, 40, 40]).cuda())
    q = torch.randn(40, 4, 64, generator=g).to(torch.bfloat16).cuda()
    sizes = [fa.fwd_paged_fp8_workspace_size(2, 4, 2, 64, 32, table.shape[1], t, t, 3) for t in (1, 40)]
    ws = e(max(sizes), dt=torch.uint8)
    run = lambda i: fa.fwd_paged_fp8(q[:(1, 40)[i]], kc, vc, ks, vs, table, n, cu[i], (1, 40)[i], num_splits=3, workspace=ws)
    want = [run(0), run(1)]
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for i in (0, 1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(run(i))
        graphs.append(gr)
    ws.fill_(255)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert fa.debug_read_status() == 0
    assert all(torch.equal(a, b) for x, y in zip(want, outs) for a, b in zip(x, y))


@pytest.mark.parametrize("B,window,sinks,extra,lq", [(1000, 64, 4, 0, 1), (1000, 0, 0, 4000, 1), (1000, 0, 0, 0, 3), (700, 0, 0, 4000, 2),
                                                     (40, 30, 17, 0, 1)])
def test_many_sequences(B, window, sinks, extra, lq):
    """More groups of rows than a block has threads, many to a share."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(B)
    P, Hq, Hkv, d = 16, 4, 2, 64
    lens = [int(n) for n in torch.randint(lq - 1 if lq == 1 else lq, 200, (B,), generator=g)]
    kc, vc, ks, vs, table, full = pool(g, lens, P, Hkv, d)
    table = torch.nn.functional.pad(table, (0, extra), value=-1)
    q = torch.randn(B * lq, Hq, d, generator=g).to(torch.bfloat16)
    kw = dict(scale=0.15, window=window, sinks=sinks)
    dev = [t.cuda() for t in (q, kc, vc, ks, vs, table, i32(lens))]
    for S in (1, 3):
        if lq == 1:
            o, lse = fa.decode_paged_fp8(*dev, S, **kw)
            lse = lse.t()
        else:
            o, lse = fa.fwd_paged_fp8(*dev, i32([lq * b for b in range(B + 1)]).cuda(), lq, num_splits=S, **kw)
        assert fa.debug_read_status() == 0
        for b in list(range(0, B, 37)) + [B - 1]:
            n, rows = lens[b], slice(b * lq, (b + 1) * lq)
            vis = R.window_with_sinks(lq, n, n - lq, True, window, sinks)
            ref = R.forward(f64(q[rows]), *full[b], 0.15, 0.0, None, vis, n - lq)
            vt = np.repeat(f64(vs[table[b, :-(-n // P)].long()]), P, 0)[:n]
            pk = peaks(f64(q[rows]), full[b][0], vt, 0.15, 0.0, None, vis, n - lq, ref[1])
            check_codes(o[rows], lse[:, rows], ref, pk, n, f"splits {S} sequence {b}")
        # and all of them against single calls' bits, a sequence at a time
        for b in range(5, B, 101):
            one = [q[b * lq:(b + 1) * lq].cuda(), *dev[1:5], table[b:b + 1].cuda(), i32(lens[b:b + 1]).cuda()]
            if lq == 1:
                o1, _ = fa.decode_paged_fp8(*one, 1, **kw)
            else:
                o1, _ = fa.fwd_paged_fp8(*one, i32([0, lq]).cuda(), lq, num_splits=1, **kw)
            if S == 1:
                assert torch.equal(o1, o[b * lq:(b + 1) * lq])
