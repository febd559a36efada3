"""Attention under any visibility mask in 64 bits, with the sums that the error bounds of the GPU tests are made of (numpy,
one sequence at a time; the scores are those of shaped_ref)."""
import numpy as np

from tests.shaped_ref import scores


def window_with_sinks(N, L, off, causal, window, sinks):
    """[N, L]: key j visible to the query at i + off."""
    i, j = np.arange(N)[:, None] + off, np.arange(L)[None]
    vis = (np.abs(i - j) < window) | (j < sinks) if window else np.ones((N, L), bool)
    return vis & (j <= i) if causal else vis


def forward(q, k, v, scale, cap, slopes, vis, off=0):
    """q [N, Hq, d], k, v [L, Hkv, d] -> O, lse [Hq, N], sum_j p |v| and the magnitude behind the scores."""
    N, Hq, d = q.shape
    Hkv = k.shape[1]
    O, A, lse, M = np.zeros((N, Hq, d)), np.zeros((N, Hq, d)), np.full((Hq, N), -np.inf), np.zeros((Hq, N))
    for h in range(Hq):
        kh, vh = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq]
        s, _, mag = scores(q[:, h], kh, scale, cap, None if slopes is None else slopes[h], off)
        s, mag = np.where(vis, s, -np.inf), np.where(vis, mag, 0.0)
        m = np.max(s, 1, initial=-np.inf)
        live = np.isfinite(m)
        p = np.where(vis, np.exp(s - np.where(live, m, 0)[:, None]), 0.0)
        l = p.sum(1)
        lse[h, live] = m[live] + np.log(l[live])
        p /= np.where(live, l, 1)[:, None]
        O[:, h], A[:, h], M[h] = p @ vh, p @ np.abs(vh), mag.max(1, initial=0)
    return O, lse, A, M


def backward(q, k, v, o, lse, do, scale, cap, slopes, vis):
    """dq, dk, dv from the given o and lse, the sums of magnitudes that their low-precision products round against, and
    the terms that the fp32 errors of P, dP and D scale with."""
    Hq, Hkv = q.shape[1], k.shape[1]
    g, a, e = ({n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v))} for _ in range(3))
    for h in range(Hq):
        kv = h * Hkv // Hq
        s, f, _ = scores(q[:, h], k[:, kv], scale, cap, None if slopes is None else slopes[h], 0)
        p = np.where(vis, np.exp(np.where(vis, s - lse[h][:, None], 0)), 0.0)
        D, Dm = (do[:, h] * o[:, h]).sum(1), np.abs(do[:, h] * o[:, h]).sum(1)
        dp, dpm = do[:, h] @ v[:, kv].T, np.abs(do[:, h]) @ np.abs(v[:, kv]).T
        ds, pm = p * f * (dp - D[:, None]), p * np.abs(f) * (dpm + Dm[:, None])
        for x, m, n, y in ((p.T, p.T, "dv", do[:, h]), (ds.T * scale, np.abs(ds).T * abs(scale), "dk", q[:, h])):
            g[n][:, kv] += x @ y
            a[n][:, kv] += m @ np.abs(y)
        g["dq"][:, h] = ds @ k[:, kv] * scale
        a["dq"][:, h] = np.abs(ds) @ np.abs(k[:, kv]) * abs(scale)
        e["dq"][:, h] = pm @ np.abs(k[:, kv]) * abs(scale)
        e["dk"][:, kv] += pm.T @ np.abs(q[:, h]) * abs(scale)
    e["dv"] = a["dv"]
    return g, a, e
