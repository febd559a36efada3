"""Workloads of the 8-bit paged cache and of windows that keep the first tokens visible.

A case is a dict of plain values. ``prepare`` makes its inputs on the GPU, ``run`` is one pass through the operator: with
``own`` false in elementary torch operations (the plain form), with ``own`` true through
``exact_tiled_attention_fattn_gb300.fattn``. ``exact`` computes the same outputs from the definitions in 64 bits.

Kinds of case:
  append8  q and k of new tokens rotated, k and v written as E4M3 codes with one scale per page and head
  decode8  attention of one token per sequence over the 8-bit cache
  chunk8   attention of query chunks over the 8-bit cache
  fwd      dense attention in a window, the first ``sinks`` tokens always visible
  bwd      its gradients
  paged    the same mask for query chunks over a bf16 cache
  decode   and for one token per sequence
"""
import math

import numpy as np
import torch

own = False
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one serving step of 64 sequences, each with a partly filled last page (latency)
        dict(name="append8_tokens", kind="append8", B=64, Lq=1, ctx=1900, Hq=32, Hkv=8, d=128, rot=128, inter=False, page=16),
        # chunks of four prompts, ragged, interleaved pairs, half of the head rotated
        dict(name="append8_prompt", kind="append8", B=4, Lq=2048, ctx=4000, Hq=32, Hkv=8, d=128, rot=64, inter=True, page=32),
        # a serving batch with long ragged contexts
        dict(name="decode8_long", kind="decode8", B=8, Lq=1, ctx=32768, Hq=32, Hkv=8, d=128, cap=0.0, slopes=False, window=0,
             sinks=0, page=16),
        # one endless conversation: a window and the first tokens (latency)
        dict(name="decode8_stream", kind="decode8", B=1, Lq=1, ctx=20001, Hq=16, Hkv=2, d=64, cap=0.0, slopes=False,
             window=1024, sinks=4, page=32),
        # chunked prompts against long contexts: the largest product
        dict(name="chunk8_prompt", kind="chunk8", B=2, Lq=2048, ctx=16384, Hq=32, Hkv=8, d=128, causal=True, cap=0.0,
             slopes=False, window=0, sinks=0, page=16),
        # a few drafted tokens per sequence are checked, capped scores
        dict(name="chunk8_verify", kind="chunk8", B=4, Lq=6, ctx=12001, Hq=32, Hkv=8, d=128, causal=True, cap=50.0,
             slopes=False, window=0, sinks=0, page=64),
        # training sequences of a model with a window and sinks
        dict(name="fwd_sinks", kind="fwd", B=2, N=8192, Hq=32, Hkv=8, d=128, causal=True, cap=0.0, slopes=False, window=2048,
             sinks=4),
        # their gradients
        dict(name="bwd_sinks", kind="bwd", B=2, N=4096, Hq=32, Hkv=8, d=128, causal=True, cap=0.0, slopes=False, window=1024,
             sinks=4),
        # a short odd sequence, both sides of the window, distance bias, d = 64
        dict(name="bwd_sinks_odd", kind="bwd", B=1, N=997, Hq=8, Hkv=2, d=64, causal=False, cap=0.0, slopes=True, window=100,
             sinks=17),
        # a short capped batch (latency)
        dict(name="fwd_sinks_short", kind="fwd", B=1, N=500, Hq=4, Hkv=4, d=64, causal=True, cap=30.0, slopes=False, window=64,
             sinks=1),
        # ragged chunks over a bf16 cache, more sinks than a tile has keys
        dict(name="paged_sinks", kind="paged", B=3, Lq=517, ctx=9000, Hq=16, Hkv=4, d=64, causal=True, cap=0.0, slopes=False,
             window=2000, sinks=130, page=16),
        # a serving batch that keeps a window and its first tokens in a bf16 cache
        dict(name="decode_sinks", kind="decode", B=8, Lq=1, ctx=32768, Hq=32, Hkv=8, d=128, cap=0.0, slopes=False, window=4096,
             sinks=64, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append8", "decode8", "chunk8", "fwd", "bwd", "paged", "decode"])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = min(hkv * rng.choice([1, 2, 4, 5, 8]), 40)
    hq -= hq % hkv
    heads = dict(Hq=hq, Hkv=hkv, d=d)
    if kind == "append8":
        lq = rng.choice([1, _log(rng, 2, 2000)])
        return dict(kind=kind, B=rng.randint(1, 64 if lq < 64 else 4), Lq=lq, ctx=lq + _log(rng, 1, 3000), **heads,
                    rot=rng.choice([d, d // 2]), inter=rng.random() < 0.5, page=page)
    always = kind in ("fwd", "bwd", "paged", "decode")       # these are windows with sinks in every case
    window = _log(rng, 16, 4096) if always or rng.random() < 0.5 else 0
    shape = dict(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3, window=window,
                 sinks=_log(rng, 1, 200) if always else rng.choice([0, _log(rng, 1, 200)]) if window else 0)
    if kind in ("fwd", "bwd"):
        return dict(kind=kind, B=rng.randint(1, 2), N=_log(rng, 3, 4096), Hq=min(hq, 32), Hkv=hkv if hq <= 32 else 1, d=d,
                    causal=rng.random() < 0.8, **shape)
    lq = 1 if kind in ("decode", "decode8") else _log(rng, 1, 1000)
    return dict(kind=kind, B=rng.randint(1, 8 if lq == 1 else 3), Lq=lq, ctx=lq + _log(rng, 5, 30000 if lq == 1 else 8000),
                **heads, **({} if lq == 1 and kind != "chunk8" and kind != "paged" else dict(causal=rng.random() < 0.8)), **shape,
                page=page)


# ---------------------------------------------------------------- shapes that follow from a case alone
def _lengths(case):
    """Context lengths of a ragged batch: sequence 0 the longest, the others shorter, down to about 45 %."""
    B, ctx, lq = case["B"], case["ctx"], case["Lq"]
    return [max(ctx - (ctx * 55 // 100) * b // B - (b % 3), lq) for b in range(B)]


def _chunks(case):
    """New tokens per sequence of a ragged chunk batch."""
    return [max(1, case["Lq"] - (case["Lq"] // 4) * (b % 3)) for b in range(case["B"])]


def _seen(case, rows, keys, off):
    """Visible pairs of one head, and the keys that any row sees."""
    i = np.arange(rows, dtype=np.int64) + off
    W, S = case["window"], case["sinks"]
    hi = np.minimum(i + 1, keys) if case.get("causal", True) else np.minimum(i + W, keys) if W else np.full(rows, keys)
    lo = np.maximum(i - W + 1, 0) if W else np.zeros(rows, np.int64)
    # sinks below the window; without causal those past its end as well
    more = np.minimum(S, lo) + (0 if case.get("causal", True) else np.maximum(np.minimum(S, keys) - hi, 0)) if W else 0
    pairs = int((hi - lo + more).sum())
    first = int(lo.min())
    return pairs, int(hi.max()) - first + (min(S, first) if W else 0)


def work(case):
    k, d, Hq, Hkv = case["kind"], case["d"], case["Hq"], case["Hkv"]
    if k == "append8":
        T = sum(_chunks(case))
        return {"bytes": T * d * (4 * Hq + 6 * Hkv) + 4 * T, "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    if k in ("fwd", "bwd"):
        rows = case["B"] * case["N"]
        pairs = case["B"] * Hq * _seen(case, case["N"], case["N"], 0)[0]
        if k == "fwd":
            return {"bytes": 4 * rows * (Hq + Hkv) * d + 4 * rows * Hq, "flops": 4 * d * pairs}
        return {"bytes": 8 * rows * (Hq + Hkv) * d + 4 * rows * Hq, "flops": 10 * d * pairs}
    each = [_seen(case, m, n, n - m) for n, m in zip(_lengths(case), _chunks(case))]
    rows, keys = sum(_chunks(case)), sum(e[1] for e in each)
    el = 1 if k in ("decode8", "chunk8") else 2
    cache = 2 * keys * Hkv * d * el + (8 * keys * Hkv // case["page"] if el == 1 else 0)
    return {"bytes": cache + 4 * rows * Hq * d + 4 * rows * Hq, "flops": 4 * d * Hq * sum(e[0] for e in each)}


# ---------------------------------------------------------------- inputs
def _pow2(a):
    """The least power of two s with a <= 448 s, at least 2^-100."""
    m, e = torch.frexp(a)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100)
    return torch.ldexp(torch.ones_like(a), torch.where(a > 0, e, torch.full_like(e, -100)))


def _quantized(x):
    """A cache's pages [pages, P, Hkv, d] as codes and scales [pages, Hkv]."""
    s = _pow2(x.abs().amax((1, 3)).float())
    return (x.float() / s[:, None, :, None]).to(E4M3), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)          # tables and the like, on the host
    gd = torch.Generator(device=dev).manual_seed(seed)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gd, device=dev) * std).to(torch.bfloat16)

    c, k = case, case["kind"]
    Hq, Hkv, d, B = c["Hq"], c["Hkv"], c["d"], c["B"]
    st = {"case": case, "scale": 1.0 / math.sqrt(d), "slopes": None}
    big = 2.0 if c.get("cap") else 1.0
    if c.get("slopes"):  # steeper heads forget faster, as a distance bias is used
        st["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=torch.float64) / Hq)).float().to(dev)
    if k in ("fwd", "bwd"):
        N = c["N"]
        st.update(q=rnd(B, N, Hq, d, std=big), k=rnd(B, N, Hkv, d, std=big), v=rnd(B, N, Hkv, d),
                  off=torch.zeros(B, dtype=torch.int64, device=dev), n=torch.full((B,), N, device=dev))
        if k == "bwd":
            st["o"], st["lse"] = _plain_dense(st)
            st["do"] = rnd(B, N, Hq, d)
        return st
    lens, chunks, P = _lengths(c), _chunks(c), c["page"]
    per = [-(-n // P) for n in lens]
    pages = sum(per) + 3                              # a shuffled pool with a few spare pages
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.zeros(B, max(per), dtype=torch.int32)
    inside = torch.arange(max(per))[None] < torch.tensor(per)[:, None]
    table[inside] = perm[:sum(per)]
    m, n = torch.tensor(chunks), torch.tensor(lens)
    i = torch.arange(max(chunks))[None]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), m.cumsum(0)])
    real = i < m[:, None]
    st.update(table=table.to(dev), seqlens=n.to(torch.int32).to(dev), cu=cu.to(torch.int32).to(dev), n=n.to(dev),
              off=(n - m).to(dev), longest=max(chunks),
              rows=torch.where(real, cu[:-1, None] + i, 0).to(dev),           # packed row of query i of sequence b
              flat=real.flatten().nonzero()[:, 0].to(dev))                    # and the way back
    T = sum(chunks)
    # keys have a few heavy channels, as keys in use do
    heavy = torch.where(torch.rand(Hkv, d, generator=gd, device=dev) < 0.03, 4.0, 1.0)
    kc, vc = (rnd(pages, P, Hkv, d, std=big).float() * heavy).to(torch.bfloat16), rnd(pages, P, Hkv, d)
    if k in ("append8", "decode8", "chunk8"):
        (kc, st["ks"]), (vc, st["vs"]) = _quantized(kc), _quantized(vc)
    st.update(kc=kc, vc=vc)
    if k == "append8":
        x = rnd(T, (Hq + 2 * Hkv) * d)                # views of one packed projection
        st.update(q=x[:, :Hq * d].view(T, Hq, d), k=x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d),
                  v=x[:, (Hq + Hkv) * d:].view(T, Hkv, d),
                  inv_freq=(10000.0 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64) / (c["rot"] // 2))).to(dev),
                  pos=(st["off"][:, None] + i.to(dev)).flatten()[st["flat"]].to(torch.int32),
                  seq=torch.repeat_interleave(torch.arange(B), m).to(dev))
        return st
    st["q"] = rnd(T, Hq, d, std=big)
    return st


# ---------------------------------------------------------------- plain forms (32 bits)
def _hidden(c, off, n, rows, keys):
    """[B, rows, keys]: what query i of sequence b does not see."""
    i = off[:, None, None] + torch.arange(rows, device=off.device)[None, :, None]
    j = torch.arange(keys, device=off.device)[None, None, :]
    hid = j >= n[:, None, None]
    if c.get("causal", True):
        hid = hid | (j > i)
    if c["window"]:
        hid = hid | (((i - j).abs() >= c["window"]) & (j >= c["sinks"]))
    return hid, (i - j).abs()


def _logits(st, q, k, hid, dist):
    """q [B, Hkv, G, N, d], k [B, Hkv, L, d] in 32 bits: scores [B, Hkv, G, N, L], -inf where hidden, and the cap's tanh."""
    c = st["case"]
    B, Hkv, G, N, d = q.shape
    s = ((q.reshape(B, Hkv, G * N, d) @ k.transpose(2, 3)) * st["scale"]).view(B, Hkv, G, N, -1)
    t = None
    if c["cap"]:
        t = torch.tanh(s / c["cap"])
        s = c["cap"] * t
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * dist[:, None, None].float()
    return s.masked_fill_(hid[:, None, None], float("-inf")), t


def _heads(x, Hkv):
    """[B, N, H, d] as [B, Hkv, G, N, d] in 32 bits."""
    B, N, H, d = x.shape
    return x.float().view(B, N, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)


def _softmax_out(s, v):
    B, Hkv, G, N, L = s.shape
    lse = torch.logsumexp(s, dim=-1)
    p = torch.exp(s - lse[..., None])
    return (p.reshape(B, Hkv, G * N, L) @ v).view(B, Hkv, G, N, -1), lse


def _attend(st, q, k, v):
    """q [B, N, Hq, d] over k, v [B, L, Hkv, d] (32 bits): o [B, N, Hq, d] bf16 and lse [B, Hq, N]."""
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    hid, dist = _hidden(st["case"], st["off"], st["n"], N, k.shape[1])
    s, _ = _logits(st, _heads(q, Hkv), k.transpose(1, 2), hid, dist)
    o, lse = _softmax_out(s, v.transpose(1, 2))
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, d).to(torch.bfloat16), lse.reshape(B, Hq, N)


def _plain_dense(st):
    return _attend(st, st["q"], st["k"].float(), st["v"].float())


def _cached(st, cache, scales):
    """The sequences' rows of a paged cache, [B, L, Hkv, d] in 32 bits, slots past a sequence's end 0."""
    pages = st["table"].long()
    x = cache[pages].float()
    if scales is not None:
        x = x * scales[pages][:, :, None, :, None]
    x = x.flatten(1, 2)
    past = torch.arange(x.shape[1], device=x.device)[None, :] >= st["n"][:, None]
    return x.masked_fill_(past[:, :, None, None], 0.0)


def _plain_paged(st):
    """Query chunks over a cache (single tokens are chunks of one): o [T, Hq, d] and lse [Hq, T]."""
    Hq, d = st["q"].shape[1:]
    o, lse = _attend(st, st["q"][st["rows"]], _cached(st, st["kc"], st.get("ks")), _cached(st, st["vc"], st.get("vs")))
    return o.reshape(-1, Hq, d)[st["flat"]], lse.transpose(0, 1).reshape(Hq, -1)[:, st["flat"]]


def _plain_bwd(st):
    q, k, v, o, do = st["q"], st["k"], st["v"], st["o"], st["do"]
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    hid, dist = _hidden(st["case"], st["off"], st["n"], N, N)
    qh, gh, kh, vh = _heads(q, Hkv), _heads(do, Hkv), k.float().transpose(1, 2), v.float().transpose(1, 2)
    s, t = _logits(st, qh, kh, hid, dist)
    p = torch.exp(s - st["lse"].view(B, Hkv, G, N, 1))
    D = (gh * _heads(o, Hkv)).sum(-1, keepdim=True)
    dp = (gh.reshape(B, Hkv, G * N, d) @ vh.transpose(2, 3)).view(B, Hkv, G, N, N)
    ds = p * (dp - D)
    if t is not None:
        ds = ds * (1 - t * t)
    flat = lambda x: x.reshape(B, Hkv, G * N, -1)
    dq = (flat(ds) @ kh * st["scale"]).view(B, Hkv, G, N, d).permute(0, 3, 1, 2, 4).reshape(q.shape)
    dk = (flat(ds).transpose(2, 3) @ flat(qh) * st["scale"]).transpose(1, 2)
    dv = (flat(p).transpose(2, 3) @ flat(gh)).transpose(1, 2)
    return dq.to(q.dtype), dk.to(k.dtype).contiguous(), dv.to(v.dtype).contiguous()


def _rotate(x, st):
    """x [T, H, d] rotated in 32 bits (angles in 64), not yet rounded."""
    r = st["case"]["rot"]
    ang = st["pos"].double()[:, None] * st["inv_freq"][None, :]
    co, si = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    y = x.float().clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if st["case"]["inter"] else (y[..., :r // 2], y[..., r // 2:r])
    a0, b0 = a.clone(), b.clone()
    a.copy_(a0 * co - b0 * si)
    b.copy_(b0 * co + a0 * si)
    return y


def _plain_append(st):
    P = st["case"]["page"]
    t = st["pos"].long()
    page, slot = st["table"][st["seq"], t // P].long(), t % P
    used = torch.unique(page)
    fresh = torch.zeros(st["kc"].shape[0], dtype=torch.bool, device=page.device)
    fresh[page[slot == 0]] = True
    kr = _rotate(st["k"], st)

    def put(cache, scales, x):
        top = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax")[used]
        old, new = scales[used], _pow2(top)
        s = torch.where(fresh[used][:, None], new, torch.maximum(old, new))
        kept = torch.where(fresh[used][:, None], torch.ones_like(s), old / s)      # (a fresh page's other slots mean nothing)
        cache[used] = (cache[used].float() * kept[:, None, :, None]).to(E4M3)
        scales[used] = s
        cache[page, slot] = (x / scales[page][:, :, None]).to(E4M3)

    put(st["kc"], st["ks"], kr)
    put(st["vc"], st["vs"], st["v"].float())
    return _rotate(st["q"], st).to(torch.bfloat16), st["kc"], st["vc"], st["ks"], st["vs"]


# ---------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    k = c["kind"]
    if not own:
        return {"append8": _plain_append, "fwd": _plain_dense, "bwd": _plain_bwd}.get(k, _plain_paged)(st)
    from exact_tiled_attention_fattn_gb300 import fattn
    if k == "append8":
        qr = fattn.rope_append_paged_fp8(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"],
                                         st["seqlens"], st["cu"], st["inv_freq"], positions=st["pos"], interleaved=c["inter"])
        return qr, st["kc"], st["vc"], st["ks"], st["vs"]
    shape = dict(scale=st["scale"], softcap=c["cap"], slopes=st["slopes"], window=c["window"], sinks=c["sinks"])
    if k == "fwd":
        return fattn.fwd_shaped(st["q"], st["k"], st["v"], causal=c["causal"], **shape)
    if k == "bwd":
        return fattn.bwd_shaped(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], causal=c["causal"], **shape)
    if k == "chunk8":
        return fattn.fwd_paged_fp8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["seqlens"], st["cu"],
                                   st["longest"], causal=c["causal"], **shape)
    if k == "paged":
        return fattn.fwd_paged_shaped(st["q"], st["kc"], st["vc"], st["table"], st["seqlens"], st["cu"], st["longest"],
                                      causal=c["causal"], **shape)
    B, Hq, d = st["q"].shape
    if "ws" not in st:  # the split count and the workspace that a serving loop keeps
        pages = st["table"].shape[1]
        if c["window"]:
            pages = min(pages, (c["window"] + c["page"] - 2) // c["page"] + 1 + -(-c["sinks"] // c["page"]))
        st["splits"] = fattn.choose_num_splits(B, c["Hkv"], pages)
        st["ws"] = torch.empty(fattn.decode_workspace_size(B, Hq, d, st["splits"]), dtype=torch.uint8, device=st["q"].device)
    if k == "decode":
        o, lse = fattn.decode_paged_shaped(st["q"], st["kc"], st["vc"], st["table"], st["seqlens"], st["splits"],
                                           workspace=st["ws"], **shape)
    else:
        o, lse = fattn.decode_paged_fp8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["seqlens"],
                                        st["splits"], workspace=st["ws"], **shape)
    return o, lse.t()


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_append(st):
    """Codes before their rounding, in units of their page's scale: what an 8-bit code stands for."""
    c = st["case"]
    r, P = c["rot"], c["page"]

    def turned(x):
        ph = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), torch.outer(st["pos"].double(), st["inv_freq"]))[:, None, :]
        x = x.double()
        if c["inter"]:
            z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2).contiguous()) * ph
            y = torch.view_as_real(z).flatten(2)
        else:
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * ph
            y = torch.cat([z.real, z.imag], -1)
        return torch.cat([y, x[..., r:]], -1)

    k, v = turned(st["k"]), st["v"].double()
    cu, lens, tab = st["cu"].tolist(), st["seqlens"].tolist(), st["table"].tolist()
    out = []
    for cache, scales, x in ((st["kc"], st["ks"], k), (st["vc"], st["vs"], v)):
        y, s = cache.double(), scales.double()
        for b, n in enumerate(lens):
            t0 = n - (cu[b + 1] - cu[b])
            for pg in range(t0 // P, -(-n // P)):
                at, a, e = tab[b][pg], max(t0, pg * P), min(n, (pg + 1) * P)
                rows = x[cu[b] + a - t0:cu[b] + e - t0]
                need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((0, 2)).clamp(min=2.0 ** -80) / 448.0)))
                if a > pg * P:
                    grown = torch.maximum(s[at], need)
                    y[at] *= (s[at] / grown)[None, :, None]
                    s[at] = grown
                else:
                    s[at] = need
                y[at, a - pg * P:e - pg * P] = rows / s[at][None, :, None]
        out.append((y, s))
    return turned(st["q"]), out[0][0], out[1][0], out[0][1], out[1][1]


def _exact_logits(c, scale, slope, q, k, first_row):
    """One head: logits of q rows (positions first_row ..) against all keys, -inf where unseen; and d logit / d raw."""
    z = torch.einsum("id,jd->ij", q, k) * scale
    grad = torch.ones_like(z)
    if c["cap"]:
        e = torch.exp(-2.0 * z.abs() / c["cap"])
        grad = 4 * e / (1 + e) ** 2
        z = c["cap"] * torch.sign(z) * (1 - e) / (1 + e)
    j = torch.arange(k.shape[0], device=q.device, dtype=torch.float64)[None, :]
    i = torch.arange(q.shape[0], device=q.device, dtype=torch.float64)[:, None] + first_row
    if slope is not None:
        z = z - slope * torch.maximum(i - j, j - i)
    seen = torch.ones_like(z, dtype=torch.bool)
    if c["window"]:
        seen = (i - j < c["window"]) & (j - i < c["window"]) | (j < c["sinks"])
    if c.get("causal", True):
        seen = seen & (j <= i)
    return torch.where(seen, z, torch.full_like(z, float("-inf"))), grad


def exact(case, seed):
    st, c, k = prepare(case, seed), case, case["kind"]
    if k == "append8":
        return _exact_append(st)
    q, Hq, Hkv = st["q"].double(), c["Hq"], c["Hkv"]
    slope = lambda h: None if st["slopes"] is None else st["slopes"][h].item()
    if k in ("fwd", "bwd"):
        N = c["N"]
        o, lse = torch.empty_like(q), torch.empty(c["B"], Hq, N, dtype=torch.float64, device=q.device)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(st["k"].double()), torch.zeros_like(st["v"].double())
        for b in range(c["B"]):
            for h in range(Hq):
                g = h * Hkv // Hq
                kh, vh = st["k"][b, :, g].double(), st["v"][b, :, g].double()
                z, gr = _exact_logits(c, st["scale"], slope(h), q[b, :, h], kh, 0)
                if k == "fwd":
                    m = z.max(-1, keepdim=True)[0]
                    e = torch.exp(z - m)
                    l = e.sum(-1, keepdim=True)
                    o[b, :, h], lse[b, h] = e @ vh / l, (m + torch.log(l))[:, 0]
                    continue
                gh, oh = st["do"][b, :, h].double(), st["o"][b, :, h].double()
                p = torch.exp(z - st["lse"][b, h].double()[:, None])
                dz = p * (gh @ vh.T - (gh * oh).sum(-1)[:, None]) * gr * st["scale"]
                dq[b, :, h] = dz @ kh
                dk[b, :, g] += dz.T @ q[b, :, h]
                dv[b, :, g] += p.T @ gh
        return (o, lse) if k == "fwd" else (dq, dk, dv)
    o, lse = torch.empty_like(q), torch.empty(Hq, q.shape[0], dtype=torch.float64, device=q.device)
    r0 = 0
    for b, (n, m) in enumerate(zip(_lengths(c), _chunks(c))):
        t = torch.arange(n, device=q.device)
        page, slot = st["table"][b, t // c["page"]].long(), t % c["page"]
        kb, vb = st["kc"][page, slot].double(), st["vc"][page, slot].double()
        if k in ("decode8", "chunk8"):
            kb, vb = kb * st["ks"][page].double()[:, :, None], vb * st["vs"][page].double()[:, :, None]
        for h in range(Hq):
            z, _ = _exact_logits(c, st["scale"], slope(h), q[r0:r0 + m, h], kb[:, h * Hkv // Hq], n - m)
            mx = z.max(-1, keepdim=True)[0]
            e = torch.exp(z - mx)
            l = e.sum(-1, keepdim=True)
            o[r0:r0 + m, h], lse[h, r0:r0 + m] = e @ vb[:, h * Hkv // Hq] / l, (mx + torch.log(l))[:, 0]
        r0 += m
    return o, lse
