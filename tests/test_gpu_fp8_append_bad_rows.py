"""Appends to the 8-bit cache with tables and lengths that do not hold: the rows concerned are skipped, in q as in the cache, the
others of the same call are written, and nothing else is."""
import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_fp8_cache import E4M3, i32, need_scale, round_e4m3
from tests.test_gpu_shaped import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,table,cu", [
    ([40], [[0, 9, 1]], [0, 30]),                                        # a page outside the pool
    ([40, 20], [[0, -1, 1], [2, 3, -5]], [0, 30, 50]),
    ([70], [[0, 1, 2]], [0, 30]),                                        # longer than its table
    ([5], [[0, 1, 2]], [0, 9]),                                          # shorter than its chunk
    ([40, 40], [[0, 1, 2], [3, 4, 5]], [0, 8, 3]),                       # offsets that decrease
    ([40, 40, 40], [[0, 1, 2], [3, 4, 5], [5, 4, 3]], [0, 8, 3, 3]),
    ([40], [[0, 1, 2]], [-4, 5]),
    ([40, 40], [[0, 1, 2], [3, 4, 5]], [0, 10, 99]),                     # past the rows
    ([2 ** 31 - 1, -2 ** 31], [[0, 1, 2], [3, 4, 5]], [0, 10, 30])])
@pytest.mark.parametrize("odd", [False, True])
def test_bad_rows(lens, table, cu, odd):
    fa = need_gpu()
    d, P, Hq, Hkv, T, pages = 64, 16, 3, 2, 50, 6
    g = torch.Generator().manual_seed(7)
    kc, vc = (torch.full((pages, P, Hkv, d), 7, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), 2.0 ** -30, device="cuda") for _ in range(2))
    x = torch.randn(T, (Hq + 2 * Hkv) * d + 1, generator=g).to(torch.bfloat16).cuda()[:, 1 if odd else 0:][:, :(Hq + 2 * Hkv) * d]
    if not odd:
        x = x.contiguous()
    q, k, v = (x[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    out = torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fa.rope_append_paged_fp8(q, k, v, kc, vc, ks, vs, i32(table).cuda(), i32(lens).cuda(), i32(cu).cuda(),
                             torch.zeros(0, dtype=torch.float64, device="cuda"), out=out)
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
    # which rows hold, and their slots
    rows, slots, fresh = [], [], {}
    for b, n in enumerate(lens):
        c0, c1 = cu[b], cu[b + 1]
        if c0 < 0 or c1 < c0 or c1 > T:
            continue
        for r in range(c0, c1):
            t = n - c1 + r
            if 0 <= t < len(table[b]) * P and 0 <= table[b][t // P] < pages:
                pg = table[b][t // P]
                rows.append(r)
                slots.append((pg, t % P))
                fresh[pg] = fresh.get(pg, False) or max(n - (c1 - c0), 0) <= t // P * P
    for codes, scales, new in ((kc, ks, k), (vc, vs, v)):
        got, got_scale, new = codes.cpu(), f64(scales), f64(new)
        same = torch.ones(pages, P, dtype=torch.bool)
        for pg in range(pages):
            mine = [(r, s) for r, (p, s) in zip(rows, slots) if p == pg]
            if not mine:
                assert (got_scale[pg] == 2.0 ** -30).all()
                continue
            s = need_scale(np.abs(new[[r for r, _ in mine]]).max((0, 2)))
            assert np.array_equal(got_scale[pg], s if fresh[pg] else np.maximum(s, 2.0 ** -30)), pg
            for r, slot in mine:
                assert np.array_equal(f64(got.view(E4M3).float())[pg, slot], round_e4m3(new[r] / s[:, None])), (pg, slot)
                same[pg, slot] = False
            if not fresh[pg]:                                  # the other slots: code 7 in steps of the new scale, nothing left of it
                other = got[pg][same[pg]]
                assert (other == 0).all()
                same[pg] = False
        assert (got[same] == 7).all()
    skipped = [r for r in range(T) if r not in rows]
    assert torch.equal(out[rows], q[rows]) and torch.isnan(out[skipped].float()).all()
