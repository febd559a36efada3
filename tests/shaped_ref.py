"""Shaped attention in 64 bits, straight from its definition, with the sums that the error
bounds of the GPU tests are made of (numpy, one sequence at a time)."""
import numpy as np


def ranges(N, L, off, causal, window, begin=None, end=None):
    """[lo, hi) of every query row."""
    i = np.arange(N) + off
    lo, hi = np.zeros(N, np.int64), np.full(N, L, np.int64)
    if causal:
        hi = np.minimum(hi, i + 1)
    if window:
        lo = np.maximum(lo, i - window + 1)
        hi = np.minimum(hi, i + window)
    if begin is not None:
        lo = np.maximum(lo, begin)
    if end is not None:
        hi = np.minimum(hi, end)
    return lo, hi


def scores(q, k, scale, cap, slope, off):
    """Scores [N, L] of one head, the cap's derivative, and the largest magnitude that enters a score."""
    s = q @ k.T * scale
    g = np.ones_like(s)
    if cap:
        t = np.tanh(s / cap)
        s, g = cap * t, 1 - t * t
    mag = np.abs(s)
    if slope is not None:
        dist = np.abs(np.arange(q.shape[0])[:, None] + off - np.arange(k.shape[0])[None])
        s = s - slope * dist
        mag = mag + np.abs(slope) * dist
    return s, g, mag


def forward(q, k, v, scale, cap=0.0, slopes=None, lo=None, hi=None, off=0):
    """q [N, Hq, d], k, v [L, Hkv, d] -> O, lse [Hq, N], sum_j p |v| and the magnitude behind the scores."""
    N, Hq, d = q.shape
    L, Hkv = k.shape[:2]
    O, A, lse, M = np.zeros((N, Hq, d)), np.zeros((N, Hq, d)), np.full((Hq, N), -np.inf), np.zeros((Hq, N))
    j = np.arange(L)
    vis = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
    for h in range(Hq):
        kh, vh = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq]
        with np.errstate(invalid="ignore", over="ignore"):
            s, _, mag = scores(q[:, h], kh, scale, cap, None if slopes is None else slopes[h], off)
        s, mag = np.where(vis, s, -np.inf), np.where(vis, mag, 0.0)
        m = np.max(s, 1, initial=-np.inf)
        any_ = np.isfinite(m)
        p = np.where(vis, np.exp(s - np.where(any_, m, 0)[:, None]), 0.0)
        l = p.sum(1)
        lse[h, any_] = m[any_] + np.log(l[any_])
        p /= np.where(any_, l, 1)[:, None]
        O[:, h], A[:, h], M[h] = p @ vh, p @ np.abs(vh), mag.max(1, initial=0)
    return O, lse, A, M


def backward(q, k, v, o, lse, do, scale, cap=0.0, slopes=None, lo=None, hi=None):
    """dq, dk, dv from the given o and lse (the formula's D and P), each with the sum of magnitudes that
    its low-precision products round against, and P |D| terms for bounds that involve o's rounding."""
    N, Hq, d = q.shape
    L, Hkv = k.shape[:2]
    g = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    a = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    e = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k))}
    j = np.arange(L)
    vis = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
    for h in range(Hq):
        kv = h * Hkv // Hq
        s, f, _ = scores(q[:, h], k[:, kv], scale, cap, None if slopes is None else slopes[h], 0)
        live = np.isfinite(lse[h])
        p = np.where(vis & live[:, None], np.exp(np.where(vis, s, 0) - np.where(live, lse[h], 0)[:, None]), 0.0)
        D = (do[:, h] * o[:, h]).sum(1)
        Dm = (np.abs(do[:, h]) * np.abs(o[:, h])).sum(1)
        dp = do[:, h] @ v[:, kv].T
        dpm = np.abs(do[:, h]) @ np.abs(v[:, kv]).T
        ds = p * f * (dp - D[:, None])
        g["dv"][:, kv] += p.T @ do[:, h]
        a["dv"][:, kv] += p.T @ np.abs(do[:, h])
        g["dq"][:, h] = ds @ k[:, kv] * scale
        a["dq"][:, h] = np.abs(ds) @ np.abs(k[:, kv]) * abs(scale)
        g["dk"][:, kv] += ds.T @ q[:, h] * scale
        a["dk"][:, kv] += np.abs(ds).T @ np.abs(q[:, h]) * abs(scale)
        pm = p * np.abs(f) * (dpm + Dm[:, None])      # what the fp32 errors of P, dP and D scale with
        e["dq"][:, h] = pm @ np.abs(k[:, kv]) * abs(scale)
        e["dk"][:, kv] += pm.T @ np.abs(q[:, h]) * abs(scale)
    e["dv"] = a["dv"]
    return g, a, e
