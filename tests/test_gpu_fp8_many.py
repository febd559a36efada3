"""Many sequences over the 8-bit cache, every one of them against 64 bits (vectorised), in one piece and in shares of the line of
steps that hold several groups of rows. Tolerances as in test_gpu_fp8_cache."""
import math

import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_fp8_cache import H, i32, pool, score_err

pytestmark = pytest.mark.gpu


def reference(q, codes, table, lens, lq, scale, window, sinks):
    """q [B, lq, Hq, d] -> O, sum p |v| [B, Hq, lq, d], lse, the magnitude behind the scores and the largest p vscale [B, Hq, lq]."""
    kc, vc, ks, vs = codes
    B, _, Hq, d = q.shape
    P, Hkv, G = kc.shape[1], kc.shape[2], Hq // kc.shape[2]
    pg = table.long().clamp(min=0)
    L = pg.shape[1] * P
    inside = torch.arange(L)[None] < lens[:, None]
    held = lambda c, s: (torch.nan_to_num(c.float()).double() * s.double()[:, None, :, None])[pg].reshape(B, L, Hkv, d)
    heads = lambda x: x.permute(0, 2, 1, 3).repeat_interleave(G, 1)                 # [B, Hq, L, d]
    k, v = heads(held(kc, ks)), heads(held(vc, vs))
    step = vs.double()[pg][:, :, None].expand(-1, -1, P, -1).reshape(B, L, Hkv).permute(0, 2, 1).repeat_interleave(G, 1)
    x = q.double().permute(0, 2, 1, 3)
    i = (lens[:, None] - lq + torch.arange(lq)[None])[:, :, None]
    j = torch.arange(L)[None, None]
    vis = inside[:, None] & (j <= i)
    if window:
        vis = vis & ((i - j < window) | (j < sinks))
    vis = vis[:, None]
    s = (x @ k.transpose(2, 3) * scale).masked_fill(~vis, -math.inf)
    mag = s.masked_fill(~vis, 0).abs().amax(-1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse.isfinite(), lse, 0.0)[..., None])
    return p @ v, p @ v.abs(), lse, mag, (p * step[:, :, None]).amax(-1)


@pytest.mark.parametrize("B,window,sinks,extra,lq", [(1000, 64, 4, 0, 1), (1000, 0, 0, 4000, 1), (1000, 0, 0, 0, 3), (700, 0, 0, 4000, 2),
                                                     (1500, 30, 17, 4000, 1), (40, 30, 17, 0, 1)])
def test_every_sequence(B, window, sinks, extra, lq):
    fa = need_gpu()
    g = torch.Generator().manual_seed(B + lq)
    P, Hq, Hkv, d = 16, 4, 2, 64
    lens = torch.randint(0 if lq == 1 else lq, 200, (B,), generator=g)
    kc, vc, ks, vs, table, _ = pool(g, lens.tolist(), P, Hkv, d)
    q = torch.randn(B * lq, Hq, d, generator=g).to(torch.bfloat16)
    O, A, lse_ref, M, peak = (t.cuda() for t in reference(q.view(B, lq, Hq, d), (kc, vc, ks, vs), table, lens, lq, 0.15, window, sinks))
    table = torch.nn.functional.pad(table, (0, extra), value=-1)
    kw = dict(scale=0.15, window=window, sinks=sinks)
    cache = [t.cuda() for t in (kc, vc, ks, vs)]

    def call(q, table, lens, S):
        o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        if lq == 1:
            lse = torch.full((B, Hq), float("nan"), device="cuda")
            fa.decode_paged_fp8(q.cuda(), *cache, table.cuda(), lens.int().cuda(), S, out=o, lse=lse, **kw)
            lse = lse.t()
        else:
            lse = torch.full((Hq, B * lq), float("nan"), device="cuda")
            fa.fwd_paged_fp8(q.cuda(), *cache, table.cuda(), lens.int().cuda(), i32(range(0, B * lq + 1, lq)).cuda(), lq, num_splits=S,
                             out=o, lse=lse, **kw)
        assert fa.debug_read_status() == 0
        return o, lse

    for S in (1, 3, 16):
        o, lse = call(q, table, lens, S)
        got = o.double().view(B, lq, Hq, d).permute(0, 2, 1, 3)
        gl = lse.double().view(Hq, B, lq).permute(1, 0, 2)
        dead = lse_ref.isneginf()
        assert torch.equal(gl.isneginf(), dead) and got.isfinite().all() and (got[dead] == 0).all(), S
        err = score_err(M)
        assert ((gl - lse_ref)[~dead].abs() <= (err + 2.0 ** -22 * lse_ref.abs())[~dead]).all(), S
        tol = H * O.abs() * 1.01 + (2.0 ** -11 + 2 * err)[..., None] * A + (2.0 ** -25 * 448 * lens.cuda()[:, None, None] * peak)[..., None]
        worst = ((got - O).abs() - tol).amax((1, 2, 3))
        assert (worst <= 0).all(), (S, int(worst.argmax()), float(worst.max()))
        if S == 1:   # a group by itself: the same bits wherever it stands in the batch
            o2, lse2 = call(q.view(B, lq, Hq, d).flip(0).reshape(-1, Hq, d), table.flip(0), lens.flip(0), 1)
            assert torch.equal(o2.view(B, lq, Hq, d).flip(0).reshape(-1, Hq, d), o)
            assert torch.equal(lse2.view(Hq, B, lq).flip(1).reshape(Hq, -1), lse.reshape(Hq, -1))
