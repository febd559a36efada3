"""The 8-bit cache with table entries outside the pool: a chunk's tokens there are zeros whether its rows are streamed or go
through the bf16 copy, a single token does not see them. Tolerances as in test_gpu_fp8_cache."""
import numpy as np
import pytest
import torch

from tests import visible_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_fp8_cache import check_codes, i32, peaks, pool
from tests.test_gpu_shaped import alibi, check_fwd, f64

pytestmark = pytest.mark.gpu


def broken(seed, lens, bad, P, Hkv, d):
    """A pool whose first page, which no sequence has, holds NaN, and a table with entries outside of it at ``bad`` ({(sequence,
    page): entry}); the values that remain, zeros there."""
    kc, vc, ks, vs, table, full = pool(torch.Generator().manual_seed(seed), lens, P, Hkv, d)
    kc, vc = (torch.cat([torch.full_like(c[:1].view(torch.uint8), 0x7f), c.view(torch.uint8)]).view(c.dtype) for c in (kc, vc))
    ks, vs = (torch.cat([torch.full_like(s[:1], float("nan")), s]) for s in (ks, vs))
    table = torch.where(table >= 0, table + 1, table)
    scale_of = [np.repeat(f64(vs[table[b, :-(-n // P)].long()]), P, 0)[:n] for b, n in enumerate(lens)]
    for (b, pi), entry in bad.items():
        table[b, pi] = entry
        for x in full[b]:
            x[pi * P:(pi + 1) * P] = 0
        scale_of[b][pi * P:(pi + 1) * P] = 1
    return kc, vc, ks, vs, table, full, scale_of


@pytest.mark.parametrize("P,Hq,Hkv,d,lk,lq,causal,cap,sl,window,sinks", [
    (16, 8, 2, 128, [300, 77], [6, 2], True, 0.0, False, 0, 0),
    (32, 4, 2, 64, [300, 100], [40, 3], False, 20.0, True, 0, 0),
    (16, 8, 2, 128, [300, 200], [60, 50], True, 0.0, True, 90, 40),               # 240 rows: the most that are streamed
    (16, 8, 2, 128, [300, 200], [61, 50], True, 0.0, True, 90, 40),               # one query more: the copy
    (64, 4, 4, 64, [400, 129], [200, 129], True, 30.0, False, 0, 0),
    (128, 6, 3, 128, [600, 130], [150, 2], False, 0.0, False, 0, 0)])
def test_chunks(P, Hq, Hkv, d, lk, lq, causal, cap, sl, window, sinks):
    fa = need_gpu()
    last = [-(-n // P) - 1 for n in lk]
    bad = {(0, 0): 99999, (0, last[0]): -3, (1, max(last[1] - 1, 0)): -2 ** 31}
    kc, vc, ks, vs, table, full, scale_of = broken(P + lq[0], lk, bad, P, Hkv, d)
    q = torch.randn(sum(lq), Hq, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lq)])
    slopes = alibi(Hq) if sl else None
    sn = None if slopes is None else f64(slopes)
    streamed = max(lq) * (Hq // Hkv) <= fa.fp8_stream_rows(Hq // Hkv)
    want = []
    for b in range(2):
        off, x = lk[b] - lq[b], f64(q[cu[b]:cu[b + 1]])
        vis = R.window_with_sinks(lq[b], lk[b], off, causal, window, sinks)
        ref = R.forward(x, *full[b], 0.15, cap, sn, vis, off)
        want.append((ref, peaks(x, full[b][0], scale_of[b], 0.15, cap, sn, vis, off, ref[1])))
    wide = [(4, torch.nn.functional.pad(table, (0, 8000), value=-1))] if streamed else []
    for S, t in ((1, table), (3, table), *wide):
        o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, sum(lq)), float("nan"), device="cuda")
        fa.fwd_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), t.cuda(), i32(lk).cuda(), i32(cu).cuda(), max(lq),
                         causal=causal, scale=0.15, softcap=cap, slopes=None if slopes is None else slopes.cuda(), window=window,
                         sinks=sinks, out=o, lse=lse, num_splits=S)
        assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
        for b in range(2):
            mine = o[cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]]
            if streamed:
                check_codes(*mine, *want[b], lk[b], f"splits {S} sequence {b}")
            else:
                check_fwd(*mine, want[b][0], f"splits {S} sequence {b}")


@pytest.mark.parametrize("P,d,lens", [(16, 128, [300, 33]), (64, 64, [200, 64])])
def test_single_tokens(P, d, lens):
    fa = need_gpu()
    Hq, Hkv = 8, 2
    bad = {(0, 1): 99999, (1, 0): -7}
    kc, vc, ks, vs, table, full, scale_of = broken(P, lens, bad, P, Hkv, d)
    q = torch.randn(2, Hq, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    for S, t in ((1, table), (4, table), (4, torch.nn.functional.pad(table, (0, 8000), value=-1))):
        o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2, Hq), float("nan"), device="cuda")
        fa.decode_paged_fp8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), t.cuda(), i32(lens).cuda(), S, scale=0.15, out=o, lse=lse)
        assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
        for b, n in enumerate(lens):
            vis = np.ones((1, n), bool)
            for (s, pi) in bad:
                if s == b:
                    vis[0, pi * P:(pi + 1) * P] = False
            x = f64(q[b:b + 1])
            ref = R.forward(x, *full[b], 0.15, 0.0, None, vis, n - 1)
            check_codes(o[b:b + 1], lse[b][:, None], ref, peaks(x, full[b][0], scale_of[b], 0.15, 0.0, None, vis, n - 1, ref[1]), n,
                        f"splits {S} sequence {b}")
