"""Chunks over the 8-bit cache past the limits of the bf16 copy: many sequences in both routes, and tables of 2^31 slots for
streamed rows. Tolerances as in test_gpu_fp8_cache."""
import numpy as np
import pytest
import torch

from tests import visible_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_fp8_cache import check_codes, held, i32, peaks
from tests.test_gpu_shaped import check_fwd, f64

pytestmark = pytest.mark.gpu


def small_pool(g, pages, P, Hkv, d):
    kc, vc = ((torch.randn(pages, P, Hkv, d, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-9, -5, (pages, Hkv), generator=g).float()) for _ in range(2))
    return kc, vc, ks, vs


@pytest.mark.parametrize("long", [2, 150])
def test_more_than_65535_sequences(long):
    """Single tokens of 70000 sequences (pages are shared: nothing is written to them), and one chunk of 2 or 150."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(long)
    B, P, Hq, Hkv, d = 70000, 16, 1, 1, 64
    kc, vc, ks, vs = small_pool(g, 40, P, Hkv, d)
    maxp = -(-long // P)
    lens, lq = torch.randint(1, P + 1, (B,), generator=g), torch.ones(B, dtype=torch.long)
    table = torch.randint(0, 40, (B, maxp), generator=g).int()
    at = 66000
    lens[at] = lq[at] = long
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lq.cumsum(0)])
    q = torch.randn(int(cu[-1]), Hq, d, generator=g).to(torch.bfloat16)
    o, lse = fa.fwd_paged_fp8(*(t.cuda() for t in (q, kc, vc, ks, vs, table, lens.int(), cu.int())), long, scale=0.15, num_splits=1)
    assert fa.debug_read_status() == 0
    for b in (0, 1, 65535, 65536, at - 1, at, at + 1, B - 1):
        n, rows = int(lens[b]), slice(int(cu[b]), int(cu[b + 1]))
        full = [held(c, s, table[b].long(), n) for c, s in ((kc, ks), (vc, vs))]
        x, off = f64(q[rows]), n - int(lq[b])
        vis = R.window_with_sinks(int(lq[b]), n, off, True, 0, 0)
        ref = R.forward(x, *full, 0.15, 0.0, None, vis, off)
        if long <= fa.fp8_stream_rows(1):
            vt = np.repeat(f64(vs[table[b].long()]), P, 0)[:n]
            check_codes(o[rows], lse[:, rows], ref, peaks(x, full[0], vt, 0.15, 0.0, None, vis, off, ref[1]), n, f"sequence {b}")
        else:
            check_fwd(o[rows], lse[:, rows], ref, f"sequence {b}")


def test_wide_tables():
    fa = need_gpu()
    g = torch.Generator().manual_seed(4)
    B, P, Hq, Hkv, d, maxp = 2, 16, 4, 2, 64, 1 << 26
    kc, vc, ks, vs = small_pool(g, 70, P, Hkv, d)
    lens, cu = [500, 1000], [0, 5, 8]
    table = torch.full((B, maxp), -1, dtype=torch.int32, device="cuda")
    pages = torch.randperm(70, generator=g)[:63].int()
    for b in range(B):
        table[b, :63] = pages.cuda()
    q = torch.randn(8, Hq, d, generator=g).to(torch.bfloat16)
    for window in (0, 200):
        o, lse = fa.fwd_paged_fp8(*(t.cuda() for t in (q, kc, vc, ks, vs)), table, i32(lens).cuda(), i32(cu).cuda(), 5, scale=0.15,
                                  window=window, sinks=4 if window else 0, num_splits=7)
        assert fa.debug_read_status() == 0
        for b, n in enumerate(lens):
            full = [held(c, s, pages.long(), n) for c, s in ((kc, ks), (vc, vs))]
            rows, lq = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
            x = f64(q[rows])
            vis = R.window_with_sinks(lq, n, n - lq, True, window, 4)
            ref = R.forward(x, *full, 0.15, 0.0, None, vis, n - lq)
            vt = np.repeat(f64(vs[pages.long()]), P, 0)[:n]
            check_codes(o[rows], lse[:, rows], ref, peaks(x, full[0], vt, 0.15, 0.0, None, vis, n - lq, ref[1]), n, f"window {window} sequence {b}")
