"""Workloads of the rotary, shaped-score and cache-eviction operators.

A case is a dict of plain values. ``prepare`` makes its inputs on the GPU, ``run`` is one
pass through the operator: with ``own`` false in elementary torch operations (the plain
form), with ``own`` true through ``exact_tiled_attention_fattn_gb300.fattn``. ``exact``
computes the same outputs from the definitions in 64 bits.

Kinds of case:
  rope     rotary positions on q and k (views of one packed projection); inverse = gradient
  append   the serving form: q and k of new tokens rotated, k and v put into their pages
  fwd      prefill with shaped scores (tanh cap, distance bias, window, key ranges)
  paged    the same for query chunks over a paged cache
  bwd      gradients of ``fwd``
  decode   the same scores for one token per sequence over a paged cache
  weights  attention weight that the cache's tokens received from the given queries
  evict    every KV head of every sequence cut down to its heaviest tokens
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # q and k of a training batch of 4 x 4096 tokens, 32 heads over 8, taken from the packed projection
        dict(name="rope_train", kind="rope", B=4, N=4096, Hq=32, Hkv=8, d=128, rot=128, inter=False, dtype="bf16",
             inverse=False, scaled=False, start=0),
        # one serving step of 64 sequences: interleaved pairs, half of the head, positions far out (latency)
        dict(name="append_tokens", kind="append", B=64, Lq=1, ctx=1900, Hq=32, Hkv=4, d=128, rot=64, inter=True,
             page=16, scaled=True, start=120000),
        # prompts of a model with capped scores and a sliding window
        dict(name="fwd_cap_window", kind="fwd", B=2, N=8192, Hq=32, Hkv=8, d=128, causal=True, cap=50.0, slopes=False,
             window=4096, doc=0, prefix=0),
        # chunked prompts of a model with a distance bias, ragged, d = 64
        dict(name="paged_bias_chunk", kind="paged", B=3, Lq=517, ctx=9000, Hq=16, Hkv=4, d=64, causal=True, cap=0.0,
             slopes=True, window=0, page=16),
        # training on packed documents with capped scores: the largest case
        dict(name="bwd_docs_cap", kind="bwd", B=4, N=4096, Hq=32, Hkv=32, d=128, causal=True, cap=30.0, slopes=False,
             window=0, doc=900, prefix=0),
        # a short odd sequence with bidirectional prefixes and a distance bias, d = 64
        dict(name="bwd_prefix_bias", kind="bwd", B=1, N=997, Hq=8, Hkv=2, d=64, causal=False, cap=0.0, slopes=True,
             window=0, doc=400, prefix=120),
        # a serving batch with long ragged contexts and capped scores
        dict(name="decode_cap_long", kind="decode", B=8, ctx=32768, Hq=32, Hkv=8, d=128, cap=50.0, slopes=False,
             window=0, page=16),
        # one sequence, window and distance bias (latency)
        dict(name="decode_window_one", kind="decode", B=1, ctx=9001, Hq=16, Hkv=2, d=64, cap=0.0, slopes=True,
             window=1024, page=32),
        # weights that one generated token per sequence adds
        dict(name="weights_tokens", kind="weights", B=8, Lq=1, ctx=16384, Hq=32, Hkv=8, d=128, cap=0.0, slopes=False,
             window=0, page=16),
        # weights from the last chunk of two prompts
        dict(name="weights_prompt", kind="weights", B=2, Lq=2048, ctx=5000, Hq=32, Hkv=8, d=128, cap=0.0, slopes=False,
             window=0, page=16),
        # a long batch cut to 4096 tokens per head
        dict(name="evict_long", kind="evict", B=8, ctx=16384, Hkv=8, d=128, keep=4096, recent=1024, first=4, page=16),
        # one short sequence (latency)
        dict(name="evict_short", kind="evict", B=1, ctx=1500, Hkv=2, d=64, keep=777, recent=100, first=0, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "fwd", "paged", "bwd", "decode", "weights", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5])
    page = rng.choice([16, 32, 64, 128])
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    slopes = rng.random() < 0.5
    window = rng.choice([0, _log(rng, 16, 4096)])
    if kind == "rope":
        return dict(kind=kind, B=rng.randint(1, 4), N=_log(rng, 1, 4096), Hq=hq, Hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), inter=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp32"]),
                    inverse=rng.random() < 0.5, scaled=rng.random() < 0.5, start=rng.choice([0, _log(rng, 10, 1000000)]))
    if kind == "append":
        lq = rng.choice([1, _log(rng, 2, 2000)])
        return dict(kind=kind, B=rng.randint(1, 64 if lq < 64 else 8), Lq=lq, ctx=lq + _log(rng, 1, 4000), Hq=hq,
                    Hkv=hkv, d=d, rot=rng.choice([d, d // 2]), inter=rng.random() < 0.5, page=page,
                    scaled=rng.random() < 0.5, start=rng.choice([0, _log(rng, 10, 1000000)]))
    if kind in ("fwd", "bwd"):
        n = _log(rng, 3, 4096)
        doc = rng.choice([0, _log(rng, 8, 2000)])
        prefix = rng.choice([0, max(1, doc // 3)]) if doc else 0
        return dict(kind=kind, B=rng.randint(1, 2), N=n, Hq=min(hq, 32), Hkv=hkv if hq <= 32 else 1, d=d,
                    causal=prefix == 0 and rng.random() < 0.7, cap=cap, slopes=slopes,
                    window=window, doc=doc, prefix=prefix) if hq <= 32 else dict(
                        kind=kind, B=1, N=n, Hq=8, Hkv=2, d=d, causal=True, cap=cap, slopes=slopes, window=window,
                        doc=0, prefix=0)
    if kind == "paged":
        lq = _log(rng, 1, 2000)
        return dict(kind=kind, B=rng.randint(1, 4), Lq=lq, ctx=lq + _log(rng, 1, 8000), Hq=hq, Hkv=hkv, d=d,
                    causal=rng.random() < 0.8, cap=cap, slopes=slopes, window=window, page=page)
    if kind == "decode":
        return dict(kind=kind, B=rng.randint(1, 8), ctx=_log(rng, 5, 30000), Hq=hq, Hkv=hkv, d=d, cap=cap,
                    slopes=slopes, window=window, page=page)
    if kind == "weights":
        lq = rng.choice([1, _log(rng, 2, 2000)])
        return dict(kind=kind, B=rng.randint(1, 4), Lq=lq, ctx=lq + _log(rng, 5, 8000), Hq=hq, Hkv=hkv, d=d, cap=cap,
                    slopes=slopes, window=window, page=page)
    ctx = _log(rng, 40, 16000)
    keep = rng.randint(10, ctx)
    recent = rng.randint(0, keep // 2)
    return dict(kind="evict", B=rng.randint(1, 8), ctx=ctx, Hkv=hkv, d=d, keep=keep, recent=recent,
                first=rng.choice([0, min(4, keep - recent)]), page=page)


# ---------------------------------------------------------------- shapes that follow from a case alone
def _lengths(case):
    """Context lengths of a ragged batch: sequence 0 the longest, the others shorter, down to about 45 %."""
    B, ctx, lq = case["B"], case["ctx"], case.get("Lq", 1)
    return [max(ctx - (ctx * 55 // 100) * b // max(B, 1) - (b % 3), lq) for b in range(B)]


def _chunks(case):
    """New tokens per sequence of a ragged chunk batch."""
    lq = case.get("Lq", 1)
    return [max(1, lq - (lq // 4) * (b % 3)) for b in range(case["B"])]


def _ranges(case):
    """Key ranges [begin, end) of every query of one row of the batch: documents of uneven
    lengths, in each of which the first ``prefix`` tokens are visible to all of it."""
    N, doc, prefix = case["N"], case["doc"], case["prefix"]
    begin, end = np.zeros(N, np.int32), np.zeros(N, np.int32)
    s, i = 0, 0
    while s < N:
        e = min(N, s + max(1, doc * (3 + 2 * (i % 3)) // 5))
        begin[s:e] = s
        end[s:e] = np.maximum(np.arange(s, e) + 1, min(e, s + prefix)) if prefix else e
        s, i = e, i + 1
    return begin, end


def _visible(case, rows, keys, off):
    """[lo, hi) of the keys that each query row sees, from causal, window and the ranges."""
    i = np.arange(rows) + off
    lo, hi = np.zeros(rows, np.int64), np.full(rows, keys, np.int64)
    W = case.get("window", 0)
    if case.get("causal", True):
        hi = np.minimum(hi, i + 1)
    elif W:
        hi = np.minimum(hi, i + W)
    if W:
        lo = np.maximum(lo, i - W + 1)
    if case.get("doc", 0):
        b, e = _ranges(case)
        lo, hi = np.maximum(lo, b), np.minimum(hi, e)
    return lo, np.maximum(hi, lo)


def work(case):
    k = case["kind"]
    if k in ("rope", "append"):
        el = 4 if case.get("dtype") == "fp32" else 2
        if k == "rope":
            T, heads = case["B"] * case["N"], case["Hq"] + case["Hkv"]
            rotated = heads
        else:
            T, heads = sum(_chunks(case)), case["Hq"] + 2 * case["Hkv"]
            rotated = case["Hq"] + case["Hkv"]
        return {"bytes": 2 * T * heads * case["d"] * el + 4 * T, "flops": 3 * T * rotated * case["rot"]}
    if k == "evict":
        keep = sum(min(case["keep"], n) for n in _lengths(case))
        row = case["Hkv"] * case["d"] * 2
        return {"bytes": 4 * keep * row + 4 * case["Hkv"] * (sum(_lengths(case)) + 2 * keep),
                "flops": case["Hkv"] * sum(_lengths(case))}
    d, Hq, Hkv, B = case["d"], case["Hq"], case["Hkv"], case["B"]
    if k in ("fwd", "bwd"):
        lo, hi = _visible(case, case["N"], case["N"], 0)
        pairs = B * Hq * int((hi - lo).sum())
        rows = B * case["N"]
        if k == "fwd":
            return {"bytes": 4 * rows * (Hq + Hkv) * d + 4 * rows * Hq, "flops": 4 * d * pairs}
        return {"bytes": 8 * rows * (Hq + Hkv) * d + 4 * rows * Hq, "flops": 10 * d * pairs}
    lens, chunks = _lengths(case), _chunks(case)
    pairs, keys = 0, 0
    for n, m in zip(lens, chunks):
        m = min(n, m)
        lo, hi = _visible(case, m, n, n - m)
        pairs += Hq * int((hi - lo).sum())
        keys += int(hi.max() - lo.min())
    rows = sum(min(n, m) for n, m in zip(lens, chunks))
    if k == "weights":
        return {"bytes": 2 * keys * Hkv * d + 2 * rows * Hq * d + 4 * rows * Hq + 8 * Hkv * sum(lens),
                "flops": 2 * d * pairs}
    return {"bytes": 4 * keys * Hkv * d + 4 * rows * Hq * d + 4 * rows * Hq, "flops": 4 * d * pairs}


# ---------------------------------------------------------------- inputs
def _frequencies(case):
    """Angles per position, radians: base 10000, or (scaled) interpolated four-fold below a band of frequencies."""
    half = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if not case["scaled"]:
        return f, 1.0
    ramp = torch.clamp(torch.arange(half, dtype=torch.float64) / max(half - 1, 1) * 2 - 0.5, 0, 1)
    return f * (1 - ramp) + f / 4 * ramp, 0.1 * math.log(4.0) + 1.0


def _pages(case, g, lens, extra=0):
    """Block table [B, max_pages] over a shuffled pool, with a few spare pages."""
    P = case["page"]
    per = [-(-n // P) for n in lens]
    maxp = max(per)
    total = sum(per) + extra + 3
    perm = torch.randperm(total, generator=g)
    table = torch.zeros(len(lens), maxp, dtype=torch.int32)
    o = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[o:o + n].to(torch.int32)
        o += n
    return table, total, perm[o:]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)          # tables and the like, on the host
    gd = torch.Generator(device=dev).manual_seed(seed)

    def rnd(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gd, device=dev) * std).to(dtype)

    k, st = case["kind"], {"case": case}
    if k in ("rope", "append"):
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        f, amp = _frequencies(case)
        st.update(inv_freq=f.to(dev), amp=amp)
        if k == "rope":
            T = case["B"] * case["N"]
            dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
            x = rnd(T, (Hq + 2 * Hkv) * d, dtype=dt)
            pos = torch.arange(case["N"], dtype=torch.int32).repeat(case["B"]) + case["start"]
            st.update(q=x[:, :Hq * d].view(T, Hq, d), k=x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d), pos=pos.to(dev))
            return st
        lens = _lengths(case)
        chunks = [min(a, b) for a, b in zip(_chunks(case), lens)]
        T = sum(chunks)
        x = rnd(T, (Hq + 2 * Hkv) * d)
        table, pages, _ = _pages(case, g, lens)
        st.update(q=x[:, :Hq * d].view(T, Hq, d), k=x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d),
                  v=x[:, (Hq + Hkv) * d:].view(T, Hkv, d), table=table.to(dev),
                  kc=rnd(pages, case["page"], Hkv, d), vc=rnd(pages, case["page"], Hkv, d),
                  seqlens=torch.tensor(lens, dtype=torch.int32, device=dev),
                  cu=torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32, device=dev),
                  pos=(torch.cat([torch.arange(n - m, n) for n, m in zip(lens, chunks)]) + case["start"]).to(
                      device=dev, dtype=torch.int32))
        return st
    if k == "evict":
        lens = _lengths(case)
        P, Hkv, d = case["page"], case["Hkv"], case["d"]
        need = [-(-min(case["keep"], n) // P) for n in lens]
        table, pages, spare = _pages(case, g, lens, extra=sum(need))
        dst = torch.zeros(len(lens), max(need), dtype=torch.int32)
        o = 0
        for b, n in enumerate(need):
            dst[b, :n] = spare[o:o + n].to(torch.int32)
            o += n
        w = torch.rand(case["B"], Hkv, table.shape[1] * P, generator=gd, device=dev) ** 4  # a few heavy tokens
        st.update(kc=rnd(pages, P, Hkv, d), vc=rnd(pages, P, Hkv, d), table=table.to(dev), dst=dst.to(dev), w=w,
                  seqlens=torch.tensor(lens, dtype=torch.int32, device=dev))
        return st
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    # steeper heads forget faster, as a distance bias is used
    slopes = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=torch.float64) / Hq)).float().to(dev) if case["slopes"] else None
    st.update(slopes=slopes, scale=1.0 / math.sqrt(d))
    if k in ("fwd", "bwd"):
        B, N = case["B"], case["N"]
        st.update(q=rnd(B, N, Hq, d, std=2.0 if case["cap"] else 1.0), k=rnd(B, N, Hkv, d, std=2.0 if case["cap"] else 1.0),
                  v=rnd(B, N, Hkv, d), begin=None, end=None)
        if case["doc"]:
            b, e = _ranges(case)
            st.update(begin=torch.from_numpy(b).to(dev).expand(B, N).contiguous(),
                      end=torch.from_numpy(e).to(dev).expand(B, N).contiguous())
        if k == "bwd":
            st["o"], st["lse"] = _plain_fwd(st)
            st["do"] = rnd(B, N, Hq, d)
        return st
    lens = _lengths(case)
    chunks = [min(a, b) for a, b in zip(_chunks(case), lens)]
    T = sum(chunks)
    table, pages, _ = _pages(case, g, lens)
    big = 2.0 if case["cap"] else 1.0
    st.update(q=rnd(T, Hq, d, std=big), kc=rnd(pages, case["page"], Hkv, d, std=big), table=table.to(dev), lens=lens,
              chunks=chunks, seqlens=torch.tensor(lens, dtype=torch.int32, device=dev),
              cu=torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32, device=dev))
    if k == "weights":
        st["w"] = torch.rand(case["B"], Hkv, table.shape[1] * case["page"], generator=gd, device=dev)
        st["vc"] = st["kc"]
        st["lse"] = _plain_paged(st)[1]
        return st
    st["vc"] = rnd(pages, case["page"], Hkv, d)
    if own and k == "decode":
        from exact_tiled_attention_fattn_gb300 import fattn
        pages = table.shape[1]                    # pages that one token can see
        if case["window"]:
            pages = min(pages, (case["window"] + case["page"] - 2) // case["page"] + 1)
        st["splits"] = fattn.choose_num_splits(case["B"], Hkv, pages)
        st["ws"] = torch.empty(fattn.decode_workspace_size(case["B"], Hq, d, st["splits"]), dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------- plain forms (32 bits)
def _rotate(x, pos, st):
    """x [T, H, d] rotated in 32 bits (angles in 64), not yet rounded."""
    c = st["case"]
    r = c["rot"]
    ang = pos.double()[:, None] * st["inv_freq"][None, :]
    if c.get("inverse"):
        ang = -ang
    co, si = (torch.cos(ang) * st["amp"]).float()[:, None, :], (torch.sin(ang) * st["amp"]).float()[:, None, :]
    y = x.float().clone()
    if c["inter"]:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * co - b * si, b * co + a * si
    else:
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * co - b * si, b * co + a * si
    return y.to(x.dtype)


def _scores(case, scale, slopes, q, k, off):
    """Shaped scores [G, rows, keys] in 32 bits of q [G, rows, d] and k [keys, d], and the tanh factor."""
    s = (q @ k.t()) * scale
    t = None
    if case["cap"]:
        t = torch.tanh(s / case["cap"])
        s = case["cap"] * t
    if slopes is not None:
        i = torch.arange(q.shape[1], device=q.device) + off
        dist = (i[:, None] - torch.arange(k.shape[0], device=q.device)[None, :]).abs().float()
        s = s - slopes[:, None, None] * dist
    return s, t


def _hidden(case, rows, keys, off, dev, begin=None, end=None):
    i = (torch.arange(rows, device=dev) + off)[:, None]
    j = torch.arange(keys, device=dev)[None, :]
    hid = torch.zeros(rows, keys, dtype=torch.bool, device=dev)
    W = case.get("window", 0)
    if case.get("causal", True):
        hid |= j > i
    if W:
        hid |= (i - j).abs() >= W
    if begin is not None:
        hid |= (j < begin[:, None]) | (j >= end[:, None])
    return hid


def _softmax_out(s, v):
    lse = torch.logsumexp(s, dim=-1)
    return torch.exp(s - lse[..., None]) @ v, lse


def _plain_fwd(st):
    c, q, k, v = st["case"], st["q"], st["k"], st["v"]
    B, N, Hq, d = q.shape
    G = Hq // k.shape[2]
    o = torch.empty_like(q)
    lse = torch.empty(B, Hq, N, device=q.device)
    for b in range(B):
        hid = _hidden(c, N, N, 0, q.device, None if st["begin"] is None else st["begin"][b],
                      None if st["begin"] is None else st["end"][b])
        for h in range(k.shape[2]):
            hs = slice(h * G, (h + 1) * G)
            s, _ = _scores(c, st["scale"], None if st["slopes"] is None else st["slopes"][hs],
                           q[b, :, hs].float().transpose(0, 1), k[b, :, h].float(), 0)
            s.masked_fill_(hid, float("-inf"))
            oh, lse[b, hs] = _softmax_out(s, v[b, :, h].float())
            o[b, :, hs] = oh.transpose(0, 1).to(o.dtype)
    return o, lse


def _plain_bwd(st):
    c, q, k, v, o, do = st["case"], st["q"], st["k"], st["v"], st["o"], st["do"]
    B, N, Hq, d = q.shape
    G = Hq // k.shape[2]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for b in range(B):
        hid = _hidden(c, N, N, 0, q.device, None if st["begin"] is None else st["begin"][b],
                      None if st["begin"] is None else st["end"][b])
        for h in range(k.shape[2]):
            hs = slice(h * G, (h + 1) * G)
            qh, kh, vh = q[b, :, hs].float().transpose(0, 1), k[b, :, h].float(), v[b, :, h].float()
            oh, gh = o[b, :, hs].float().transpose(0, 1), do[b, :, hs].float().transpose(0, 1)
            s, t = _scores(c, st["scale"], None if st["slopes"] is None else st["slopes"][hs], qh, kh, 0)
            p = torch.exp(s - st["lse"][b, hs][..., None]).masked_fill(hid, 0.0)
            dv[b, :, h] = (p.transpose(1, 2) @ gh).sum(0).to(dv.dtype)
            ds = p * (gh @ vh.t() - (gh * oh).sum(-1, keepdim=True))
            if t is not None:
                ds = ds * (1 - t * t)
            dq[b, :, hs] = (ds @ kh * st["scale"]).transpose(0, 1).to(dq.dtype)
            dk[b, :, h] = ((ds.transpose(1, 2) @ qh).sum(0) * st["scale"]).to(dk.dtype)
    return dq, dk, dv


def _gather(cache, table, b, n):
    P = cache.shape[1]
    t = torch.arange(n, device=cache.device)
    return cache[table[b, t // P].long(), t % P]          # [n, Hkv, d]


def _plain_paged(st):
    """Query chunks over the cache: o [T, Hq, d] and lse [Hq, T]; also the single-token form."""
    c, q = st["case"], st["q"]
    T, Hq, d = q.shape
    Hkv = st["kc"].shape[2]
    G = Hq // Hkv
    o, lse = torch.empty_like(q), torch.empty(Hq, T, device=q.device)
    r0 = 0
    for b, (n, m) in enumerate(zip(st["lens"], st["chunks"])):
        kb, vb = _gather(st["kc"], st["table"], b, n).float(), _gather(st["vc"], st["table"], b, n).float()
        hid = _hidden(c, m, n, n - m, q.device)
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            s, _ = _scores(c, st["scale"], None if st["slopes"] is None else st["slopes"][hs],
                           q[r0:r0 + m, hs].float().transpose(0, 1), kb[:, h], n - m)
            s.masked_fill_(hid, float("-inf"))
            oh, lse[hs, r0:r0 + m] = _softmax_out(s, vb[:, h])
            o[r0:r0 + m, hs] = oh.transpose(0, 1).to(o.dtype)
        r0 += m
    return o, lse


def _plain_weights(st):
    c, q = st["case"], st["q"]
    Hkv = st["kc"].shape[2]
    G = q.shape[1] // Hkv
    out = torch.zeros_like(st["w"])
    r0 = 0
    for b, (n, m) in enumerate(zip(st["lens"], st["chunks"])):
        kb = _gather(st["kc"], st["table"], b, n).float()
        hid = _hidden(c, m, n, n - m, q.device)
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            s, _ = _scores(c, st["scale"], None if st["slopes"] is None else st["slopes"][hs],
                           q[r0:r0 + m, hs].float().transpose(0, 1), kb[:, h], n - m)
            p = torch.exp(s - st["lse"][hs, r0:r0 + m][..., None]).masked_fill(hid, 0.0)
            out[b, h, :n] = 0.9 * st["w"][b, h, :n] + p.sum((0, 1))
        r0 += m
    return out


def _plain_append(st):
    c = st["case"]
    qr = _rotate(st["q"], st["pos"], st)
    kr = _rotate(st["k"], st["pos"], st)
    P = c["page"]
    T = qr.shape[0]
    row = torch.arange(T, device=qr.device)
    b = torch.searchsorted(st["cu"][1:].contiguous(), row, right=True)
    t = st["seqlens"][b] - st["cu"][b + 1] + row
    page, slot = st["table"][b, t // P].long(), t % P
    st["kc"][page, slot] = kr
    st["vc"][page, slot] = st["v"]
    return qr, st["kc"], st["vc"]


def _plain_evict(st):
    c, w = st["case"], st["w"]
    P, Hkv, keep = c["page"], c["Hkv"], c["keep"]
    dev = w.device
    lens = _lengths(c)
    cap = st["dst"].shape[1] * P
    new_w = torch.zeros(c["B"], Hkv, cap, device=dev)
    kept = torch.full((c["B"], Hkv, keep), -1, dtype=torch.int32, device=dev)
    for b, n in enumerate(lens):
        m = min(keep, n)
        slot = torch.arange(m, device=dev)
        for h in range(Hkv):
            x = w[b, h, :n].clone()
            x[:c["first"]] = float("inf")
            x[n - c["recent"]:] = float("inf")
            idx = torch.sort(torch.sort(x, descending=True, stable=True)[1][:m])[0]
            kept[b, h, :m] = idx.to(torch.int32)
            new_w[b, h, :m] = w[b, h, idx]
            src, dst = st["table"][b, idx // P].long(), st["dst"][b, slot // P].long()
            st["kc"][dst, slot % P, h] = st["kc"][src, idx % P, h]
            st["vc"][dst, slot % P, h] = st["vc"][src, idx % P, h]
    return st["kc"], st["vc"], torch.clamp(st["seqlens"], max=keep), new_w, kept


# ---------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    k = c["kind"]
    if not own:
        if k == "rope":
            return _rotate(st["q"], st["pos"], st), _rotate(st["k"], st["pos"], st)
        return {"append": _plain_append, "fwd": _plain_fwd, "paged": _plain_paged, "bwd": _plain_bwd,
                "decode": _plain_paged, "weights": _plain_weights, "evict": _plain_evict}[k](st)
    from exact_tiled_attention_fattn_gb300 import fattn
    if k == "rope":
        return fattn.rope(st["q"], st["k"], st["inv_freq"], positions=st["pos"], interleaved=c["inter"],
                          amplitude=st["amp"], inverse=c["inverse"])
    if k == "append":
        qr = fattn.rope_append_paged(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["table"], st["seqlens"], st["cu"],
                                     st["inv_freq"], positions=st["pos"], interleaved=c["inter"], amplitude=st["amp"])
        return qr, st["kc"], st["vc"]
    if k == "evict":
        n, w, kept = fattn.evict_paged(st["kc"], st["vc"], st["table"], st["seqlens"], st["w"], c["keep"],
                                       recent=c["recent"], first=c["first"], dst_table=st["dst"])
        return st["kc"], st["vc"], n, w, kept
    shape = dict(softcap=c["cap"], slopes=st["slopes"], window=c["window"])
    if k == "fwd":
        return fattn.fwd_shaped(st["q"], st["k"], st["v"], causal=c["causal"], scale=st["scale"], key_begin=st["begin"],
                                key_end=st["end"], **shape)
    if k == "bwd":
        return fattn.bwd_shaped(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], causal=c["causal"],
                                scale=st["scale"], key_begin=st["begin"], key_end=st["end"], **shape)
    if k == "paged":
        return fattn.fwd_paged_shaped(st["q"], st["kc"], st["vc"], st["table"], st["seqlens"], st["cu"],
                                      max(st["chunks"]), causal=c["causal"], scale=st["scale"], **shape)
    if k == "decode":
        o, lse = fattn.decode_paged_shaped(st["q"], st["kc"], st["vc"], st["table"], st["seqlens"], st["splits"],
                                           scale=st["scale"], workspace=st["ws"], **shape)
        return o, lse.t()
    return fattn.key_weights_paged(st["q"], st["kc"], st["table"], st["seqlens"], st["cu"], max(st["chunks"]), st["lse"],
                                   weights=st["w"], decay=0.9, scale=st["scale"], **shape)


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_rotate(x, st):
    """Pairs as complex numbers times amplitude * e^{i angle}."""
    c = st["case"]
    r, T = c["rot"], x.shape[0]
    turn = torch.outer(st["pos"].double(), st["inv_freq"]) * (-1.0 if c.get("inverse") else 1.0)
    ph = torch.polar(torch.full_like(turn, st["amp"]), turn)[:, None, :]
    x = x.double()
    rot, rest = x[..., :r], x[..., r:]
    if c["inter"]:
        z = torch.view_as_complex(rot.reshape(T, -1, r // 2, 2).contiguous()) * ph
        y = torch.view_as_real(z).reshape(T, -1, r)
    else:
        z = torch.complex(rot[..., :r // 2], rot[..., r // 2:]) * ph
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, rest], -1)


def _exact_logits(case, scale, slope, q, k, lo, hi, first_row):
    """One head: logits of q rows (positions first_row ..) against all keys, -inf outside [lo, hi); and d logit / d raw."""
    z = torch.einsum("id,jd->ij", q, k) * scale
    grad = torch.ones_like(z)
    if case["cap"]:
        e = torch.exp(-2.0 * z.abs() / case["cap"])
        th = torch.sign(z) * (1 - e) / (1 + e)
        grad = 4 * e / (1 + e) ** 2
        z = case["cap"] * th
    j = torch.arange(k.shape[0], device=q.device, dtype=torch.float64)
    i = torch.arange(q.shape[0], device=q.device, dtype=torch.float64) + first_row
    if slope is not None:
        z = z - float(slope) * torch.maximum(i[:, None] - j, j - i[:, None])
    seen = (j >= torch.as_tensor(lo, device=q.device)[:, None]) & (j < torch.as_tensor(hi, device=q.device)[:, None])
    return torch.where(seen, z, torch.full_like(z, float("-inf"))), grad


def exact(case, seed):
    st = prepare(case, seed)
    c, k = case, case["kind"]
    if k == "rope":
        return _exact_rotate(st["q"], st), _exact_rotate(st["k"], st)
    if k == "append":
        kc, vc = st["kc"].double(), st["vc"].double()
        kr = _exact_rotate(st["k"], st)
        cu, tab = st["cu"].tolist(), st["table"].tolist()
        pg, sl = [], []
        for b, n in enumerate(st["seqlens"].tolist()):
            for t in range(n - (cu[b + 1] - cu[b]), n):
                pg.append(tab[b][t // c["page"]])
                sl.append(t % c["page"])
        pg, sl = torch.tensor(pg, device=kc.device), torch.tensor(sl, device=kc.device)
        kc[pg, sl], vc[pg, sl] = kr, st["v"].double()
        return _exact_rotate(st["q"], st), kc, vc
    if k == "evict":
        kc, vc = st["kc"], st["vc"]
        wn = st["w"].double().cpu().numpy()
        P, lens = c["page"], _lengths(c)
        new_w = np.zeros((c["B"], c["Hkv"], st["dst"].shape[1] * P))
        kept = np.full((c["B"], c["Hkv"], c["keep"]), -1, np.int64)
        tab, dst = st["table"].cpu().numpy(), st["dst"].cpu().numpy()
        k2, v2 = kc.clone(), vc.clone()
        for b, n in enumerate(lens):
            m = min(n, c["keep"])
            always = [t for t in range(n) if t < c["first"] or t >= n - c["recent"]] if m < n else list(range(n))
            for h in range(c["Hkv"]):
                rest = np.setdiff1d(np.arange(n), always, assume_unique=True)
                rest = rest[np.lexsort((rest, -wn[b, h, rest]))][:m - len(always)]
                ids = np.sort(np.concatenate([np.array(always, np.int64), rest]))
                kept[b, h, :m], new_w[b, h, :m] = ids, wn[b, h, ids]
                s = np.arange(m)
                a = [torch.from_numpy(np.asarray(z, np.int64)).to(kc.device)
                     for z in (dst[b, s // P], s % P, tab[b, ids // P], ids % P)]
                k2[a[0], a[1], h], v2[a[0], a[1], h] = kc[a[2], a[3], h], vc[a[2], a[3], h]
        dev = kc.device
        return (k2.double(), v2.double(), torch.tensor([min(n, c["keep"]) for n in lens], device=dev),
                torch.from_numpy(new_w).to(dev), torch.from_numpy(kept).to(dev))
    slope = lambda h: None if st["slopes"] is None else st["slopes"][h].item()
    q = st["q"].double()
    if k in ("fwd", "bwd"):
        B, N, Hq, d = q.shape
        Hkv = c["Hkv"]
        lo, hi = _visible(c, N, N, 0)
        if k == "fwd":
            o, lse = torch.empty_like(q), torch.empty(B, Hq, N, dtype=torch.float64, device=q.device)
        else:
            dq, dk, dv = torch.zeros_like(q), torch.zeros_like(st["k"].double()), torch.zeros_like(st["v"].double())
        for b in range(B):
            for h in range(Hq):
                kh, vh = st["k"][b, :, h * Hkv // Hq].double(), st["v"][b, :, h * Hkv // Hq].double()
                z, gr = _exact_logits(c, st["scale"], slope(h), q[b, :, h], kh, lo, hi, 0)
                if k == "fwd":
                    m = z.max(-1, keepdim=True)[0]
                    e = torch.exp(z - m)
                    l = e.sum(-1, keepdim=True)
                    o[b, :, h] = e @ vh / l
                    lse[b, h] = (m + torch.log(l))[:, 0]
                    continue
                gh, oh = st["do"][b, :, h].double(), st["o"][b, :, h].double()
                p = torch.exp(z - st["lse"][b, h].double()[:, None])
                dv[b, :, h * Hkv // Hq] += p.T @ gh
                dz = p * (gh @ vh.T - (gh * oh).sum(-1)[:, None]) * gr * st["scale"]
                dq[b, :, h] = dz @ kh
                dk[b, :, h * Hkv // Hq] += dz.T @ q[b, :, h]
        return (o, lse) if k == "fwd" else (dq, dk, dv)
    T, Hq, d = q.shape
    Hkv = c["Hkv"]
    o, lse = torch.empty_like(q), torch.empty(Hq, T, dtype=torch.float64, device=q.device)
    w = torch.zeros_like(st["w"].double()) if k == "weights" else None
    r0 = 0
    for b, (n, m) in enumerate(zip(st["lens"], st["chunks"])):
        ids = torch.tensor([[int(p), s] for p in st["table"][b].tolist() for s in range(c["page"])][:n], device=q.device)
        kb, vb = st["kc"][ids[:, 0], ids[:, 1]].double(), st["vc"][ids[:, 0], ids[:, 1]].double()
        lo, hi = _visible(c, m, n, n - m)
        if k == "weights":
            w[b, :, :n] = 0.9 * st["w"][b, :, :n].double()
        for h in range(Hq):
            z, _ = _exact_logits(c, st["scale"], slope(h), q[r0:r0 + m, h], kb[:, h * Hkv // Hq], lo, hi, n - m)
            if k == "weights":
                w[b, h * Hkv // Hq, :n] += torch.exp(z - st["lse"][h, r0:r0 + m].double()[:, None]).sum(0)
                continue
            mx = z.max(-1, keepdim=True)[0]
            e = torch.exp(z - mx)
            l = e.sum(-1, keepdim=True)
            o[r0:r0 + m, h] = e @ vb[:, h * Hkv // Hq] / l
            lse[h, r0:r0 + m] = (mx + torch.log(l))[:, 0]
        r0 += m
    return w if k == "weights" else (o, lse)
