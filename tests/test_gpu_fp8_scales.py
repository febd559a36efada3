"""The 8-bit cache with the largest and the smallest scales. Tolerances as in test_gpu_fp8_cache."""
import numpy as np
import pytest
import torch

from tests import visible_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_fp8_cache import E4M3, check_codes, held, i32, peaks, pool, round_e4m3
from tests.test_gpu_shaped import f64

pytestmark = pytest.mark.gpu


def test_append_to_a_page_of_the_largest_scale():
    """Scales of 2^127 (its reciprocal is no normal number): values of that size keep their codes, infinities become NaN."""
    fa = need_gpu()
    kc, vc = (torch.zeros(2, 16, 1, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((2, 1), 2.0 ** 127, device="cuda") for _ in range(2))
    x = (torch.randn(2, 1, 64, generator=torch.Generator().manual_seed(1)) * 1e38).clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    x[1, 0, 3], x[1, 0, 4], x[1, 0, 5] = float("inf"), float("nan"), 2.0 ** 127
    y = x.flip(2)
    fa.rope_append_paged_fp8(None, x.cuda(), y.cuda(), kc, vc, ks, vs, i32([[1]]).cuda(), i32([7]).cuda(), i32([0, 2]).cuda(),
                             torch.zeros(0, dtype=torch.float64, device="cuda"))
    assert fa.debug_read_status() == 0 and (ks == 2.0 ** 127).all() and (vs == 2.0 ** 127).all()
    for codes, v in ((kc, x), (vc, y)):
        got, v = f64(codes.cpu().view(E4M3).float())[1, 5:7, 0], f64(v)[:, 0]
        odd = ~np.isfinite(v)
        assert np.isnan(got[odd]).all() and np.array_equal(got[~odd], round_e4m3(v[~odd] / 2.0 ** 127)) and (got[~odd] != 0).any()
        assert (codes[0] == 0).all() and (codes[1, :5] == 0).all() and (codes[1, 7:] == 0).all()


@pytest.mark.parametrize("exponent", [127, 126, 120, 60, -60, -100])
@pytest.mark.parametrize("lq", [1, 6])
def test_attention(exponent, lq):
    """V's scales around 2^exponent, codes of at most 1."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(3)
    lens, P, Hq, Hkv, d = [700, 33], 16, 8, 2, 128
    kc, vc, ks, vs, table, _ = pool(g, lens, P, Hkv, d)
    nan = vc.view(torch.uint8) == 0x7f
    vc = (vc.float() / 448).to(E4M3)
    vc.view(torch.uint8)[nan] = 0x7f
    vs = torch.exp2(torch.randint(exponent - 2 if exponent > 0 else exponent, exponent + 1 if exponent > 0 else exponent + 3, vs.shape, generator=g).float())
    full = [[held(c, s, table[b, :-(-n // P)].long(), n) for c, s in ((kc, ks), (vc, vs))] for b, n in enumerate(lens)]
    q = torch.randn(2 * lq, Hq, d, generator=g).to(torch.bfloat16)
    dev = [t.cuda() for t in (q, kc, vc, ks, vs)]
    for S, t in ((1, table), (5, table), (5, torch.nn.functional.pad(table, (0, 8000), value=-1))):
        if lq == 1:
            o, lse = fa.decode_paged_fp8(*dev, t.cuda(), i32(lens).cuda(), S, scale=0.15)
            lse = lse.t()
        else:
            o, lse = fa.fwd_paged_fp8(*dev, t.cuda(), i32(lens).cuda(), i32([0, lq, 2 * lq]).cuda(), lq, scale=0.15, num_splits=S)
        assert fa.debug_read_status() == 0
        for b, n in enumerate(lens):
            rows = slice(b * lq, (b + 1) * lq)
            vis = R.window_with_sinks(lq, n, n - lq, True, 0, 0)
            x = f64(q[rows])
            ref = R.forward(x, *full[b], 0.15, 0.0, None, vis, n - lq)
            vt = np.repeat(f64(vs[table[b, :-(-n // P)].long()]), P, 0)[:n]
            check_codes(o[rows], lse[:, rows], ref, peaks(x, full[b][0], vt, 0.15, 0.0, None, vis, n - lq, ref[1]), n, f"splits {S} sequence {b}")
