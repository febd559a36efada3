"""NaN codes in the 8-bit cache stay in their own sequence: the other sequences of a call keep their bits, in streamed rows (line of
steps, clusters, one piece), through the bf16 copy, and for single tokens."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_fp8_cache import i32, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lq", [1, 7, 200])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 5)])
def test_nan_stays_in_its_sequence(lq, window, sinks):
    fa = need_gpu()
    g = torch.Generator().manual_seed(lq)
    lens, P, Hq, Hkv, d = [400, 300, 210], 16, 8, 2, 128
    kc, vc, ks, vs, table, _ = pool(g, lens, P, Hkv, d)
    q = torch.randn(3 * lq, Hq, d, generator=g).to(torch.bfloat16).cuda()
    bad_k, bad_v = kc.clone(), vc.clone()
    page = int(table[1, (lens[1] - 1) // P])
    slot = (lens[1] - 1) % P                                   # the second sequence's last token, KV head 0
    bad_k.view(torch.uint8)[page, slot, 0, 3], bad_v.view(torch.uint8)[page, slot, 0, 5] = 0x7f, 0xff
    wide = torch.nn.functional.pad(table, (0, 8000), value=-1)
    for S, t in ((1, table), (4, table), (4, wide)) if lq < 200 else ((1, table), (3, table)):
        got = []
        for k, v in ((kc, vc), (bad_k, vc), (kc, bad_v)):
            args = (q, k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), t.cuda(), i32(lens).cuda())
            if lq == 1:
                o, lse = fa.decode_paged_fp8(*args, S, scale=0.15, window=window, sinks=sinks)
                lse = lse.t()
            else:
                o, lse = fa.fwd_paged_fp8(*args, i32([0, lq, 2 * lq, 3 * lq]).cuda(), lq, scale=0.15, window=window, sinks=sinks,
                                          num_splits=S)
            assert fa.debug_read_status() == 0
            got.append((o.float(), lse))
        good, with_k, with_v = got
        for o, lse in (with_k, with_v):
            for rows in (slice(0, lq), slice(2 * lq, 3 * lq)):
                assert torch.equal(o[rows], good[0][rows]) and torch.equal(lse[:, rows], good[1][:, rows])
            assert torch.equal(o[:, Hq // Hkv:], good[0][:, Hq // Hkv:]) and torch.equal(lse[Hq // Hkv:], good[1][Hq // Hkv:])
        last = 2 * lq - 1                                      # the row that sees the token, in KV head 0
        assert torch.isnan(with_v[0][last, :Hq // Hkv, 5]).all() and torch.isnan(with_k[1][:Hq // Hkv, last]).all()
        others = [e for e in range(d) if e != 5]
        assert torch.equal(with_v[0][:, :, others], good[0][:, :, others]) and torch.equal(with_v[1], good[1])
        before = slice(lq, last)                               # a NaN key is hidden from the rows before it
        assert torch.equal(with_k[0][before], good[0][before]) and torch.equal(with_k[1][:, before], good[1][:, before])
