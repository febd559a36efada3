"""Tanh caps far above the scores, and single scores as large as the cap among small ones, in every call that takes a cap.

Tolerance: c tanh(s / c) keeps a score's relative precision whatever c is. Besides the fp32 product, whose error the
shaped tests bound by 5e-5 + 1e-6 M with M the largest magnitude behind a row's scores, the cap may add its own 8e-8
and six roundings of 2^-24, 4.4e-7 M: inside that bound, with no term in c. Scores near -c (weight 0) do not count in M.
"""
import math

import numpy as np
import pytest
import torch

from tests import shaped_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_eviction import i32, pool, rows, weights_ref
from tests.test_gpu_shaped import H, alibi, check_fwd, f64, make, score_err

pytestmark = pytest.mark.gpu
CAPS = [300.0, 1e4, 1e6, 1e9, 1e18, 3e38]
dev = lambda t: None if t is None else t.cuda()


def outliers(q, k, cap, scale):
    """q [.., d], k [L, .., d] with keys 5, 42, 79, ... at a score of about -0.9 cap for every query; the same without them."""
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    plain = k.clone()
    plain[5::37] = 0.0
    k[5::37] = 0.0
    k[5::37, ..., 0] = -cap * math.atanh(0.9) / (4.0 * scale)
    return plain


@pytest.mark.parametrize("d,bias", [(128, False), (64, True)])
@pytest.mark.parametrize("cap,far", [(c, False) for c in CAPS] + [(300.0, True), (1e4, True), (1e6, True)])
def test_forward_and_gradient(cap, far, d, bias):
    fa = need_gpu()
    N, Hq, Hkv, scale = 300, 4, 2, 1 / math.sqrt(d)
    q, k, v, do = make(d, 1, N, Hq, Hkv, d)
    plain = outliers(q, k[0], cap, scale) if far else k[0]
    slopes = alibi(Hq) if bias else None
    kw = dict(causal=True, softcap=cap, slopes=dev(slopes))
    o, lse = fa.fwd_shaped(dev(q), dev(k), dev(v), **kw)
    got = dict(zip(("dq", "dk", "dv"), fa.bwd_shaped(dev(q), dev(k), dev(v), o, lse, dev(do), **kw)))
    assert fa.debug_read_status() == 0
    lo, hi = R.ranges(N, N, 0, True, 0)
    s = None if slopes is None else f64(slopes)
    ref = R.forward(f64(q[0]), f64(k[0]), f64(v[0]), scale, cap, s, lo, hi)
    M = R.forward(f64(q[0]), f64(plain), f64(v[0]), scale, cap, s, lo, hi)[3]
    check_fwd(o[0], lse[0], (*ref[:3], M), f"cap {cap}")
    g, a, e = R.backward(f64(q[0]), f64(k[0]), f64(v[0]), f64(o[0]), f64(lse[0]), f64(do[0]), scale, cap, s, lo, hi)
    for n in got:
        tol = H * 1.02 * (a[n] + np.abs(g[n])) + 2 * score_err(M.max()) * e[n] + 1e-30
        assert (np.abs(f64(got[n][0]) - g[n]) <= tol).all(), (n, (np.abs(f64(got[n][0]) - g[n]) / tol).max())


@pytest.mark.parametrize("lq,S", [(1, 3), (40, 1), (40, 3)])     # single tokens, a chunk, its keys in runs
@pytest.mark.parametrize("cap,far", [(c, False) for c in CAPS] + [(1e4, True), (1e6, True)])
def test_over_pages(cap, far, lq, S):
    fa = need_gpu()
    Hq, Hkv, d, P, n, scale = 8, 2, 64, 16, 700, 0.125
    kc, vc, table, _, g = pool(7, [n], P, Hkv, d)
    q = torch.randn(lq, Hq, d, generator=g).to(torch.bfloat16)
    k, v = rows(kc, table, 0, n), rows(vc, table, 0, n)
    plain = outliers(q, k, cap, scale) if far else k
    t = np.arange(n)
    kc[table[0, t // P].long(), torch.from_numpy(t % P)] = k
    args = (dev(q), dev(kc), dev(vc), dev(table), i32([n]))
    if lq == 1:
        o, lse = fa.decode_paged_shaped(*args, S, softcap=cap)
        lse = lse.t()
    else:
        o, lse = fa.fwd_paged_shaped(*args, i32([0, lq]), lq, softcap=cap, num_splits=S)
    assert fa.debug_read_status() == 0
    lo, hi = R.ranges(lq, n, n - lq, True, 0)
    ref = R.forward(f64(q), f64(k), f64(v), scale, cap, None, lo, hi, off=n - lq)
    M = R.forward(f64(q), f64(plain), f64(v), scale, cap, None, lo, hi, off=n - lq)[3]
    check_fwd(o, lse, (*ref[:3], M), f"cap {cap}")


@pytest.mark.parametrize("P,lq", [(16, 1), (16, 4), (16, 40), (3, 40)])   # streaming (8 and 32 rows), tensor cores, mma.sync
@pytest.mark.parametrize("cap,far", [(c, False) for c in CAPS] + [(1e4, True), (1e6, True)])
def test_key_weights(cap, far, P, lq):
    """A weight's bound: twice a score's and its lse's (here rounded from 64 bits), and 2^-24 per term of the sum."""
    fa = need_gpu()
    Hq, Hkv, d, n, scale = 8, 1, 64, 300, 0.125
    kc, _, table, _, g = pool(9, [n], P, Hkv, d, fill=0)
    q = torch.randn(lq, Hq, d, generator=g).to(torch.bfloat16)
    k = rows(kc, table, 0, n)
    plain = outliers(q, k, cap, scale) if far else k
    t = np.arange(n)
    kc[table[0, t // P].long(), torch.from_numpy(t % P)] = k
    lo, hi = R.ranges(lq, n, n - lq, True, 0)
    L = R.forward(f64(q), f64(k), f64(k), scale, cap, None, lo, hi, off=n - lq)[1]
    lse = torch.from_numpy(L).float()
    out = fa.key_weights_paged(dev(q), dev(kc), dev(table), i32([n]), i32([0, lq]), lq, dev(lse), softcap=cap)
    assert fa.debug_read_status() == 0
    want, _ = weights_ref(f64(q), f64(k), f64(lse), scale, cap, None, lo, hi, n - lq)
    _, mag = weights_ref(f64(q), f64(plain), f64(lse), scale, cap, None, lo, hi, n - lq)
    tol = (1.1e-4 + 2e-6 * mag + lq * Hq * 2.0 ** -24) * want + 1e-30
    got = f64(out[0, :, :n])
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("N,Hq,Hkv,d,causal,scale", [(16, 7, 1, 128, True, 0.3), (47, 9, 3, 64, False, 0.3), (300, 2, 1, 128, True, -0.3)])
def test_gradient_of_saturated_scores(N, Hq, Hkv, d, causal, scale):
    """Scores six to nine times the cap, positive ones in every other row, negative ones in the rest: the cap's derivative,
    here 1e-5 to 1e-7, keeps its relative precision (a score's error of 1e-6 of itself moves it by 2 / cap times that,
    2e-5: inside the gradients' bound)."""
    fa = need_gpu()
    cap = 5.0
    q, k, v, do = (x * s for x, s in zip(make(N, 1, N, Hq, Hkv, d), (0.25, 0.25, 1, 1)))
    q[..., 0] = 8.0 * (1 - 2 * (torch.arange(N) % 2))[:, None]
    k[..., 0] = (torch.linspace(6, 9, N) * cap / (8.0 * scale))[torch.randperm(N, generator=torch.Generator().manual_seed(N))][:, None]
    kw = dict(causal=causal, softcap=cap, scale=scale)
    o, lse = fa.fwd_shaped(dev(q), dev(k), dev(v), **kw)
    got = dict(zip(("dq", "dk", "dv"), fa.bwd_shaped(dev(q), dev(k), dev(v), o, lse, dev(do), **kw)))
    assert fa.debug_read_status() == 0
    lo, hi = R.ranges(N, N, 0, causal, 0)
    ref = R.forward(f64(q[0]), f64(k[0]), f64(v[0]), scale, cap, None, lo, hi)
    check_fwd(o[0], lse[0], ref)
    g, a, e = R.backward(f64(q[0]), f64(k[0]), f64(v[0]), f64(o[0]), f64(lse[0]), f64(do[0]), scale, cap, None, lo, hi)
    for n in got:
        tol = H * 1.02 * (a[n] + np.abs(g[n])) + 2 * score_err(ref[3].max()) * e[n] + 1e-30
        assert (np.abs(f64(got[n][0]) - g[n]) <= tol).all(), (n, (np.abs(f64(got[n][0]) - g[n]) / tol).max())
