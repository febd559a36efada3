"""Rotary positions and the paged append against a plain 64-bit computation.

Tolerance: angle, sine and cosine carry at most about 4 fp32 steps (the angle's 2^-25 of a turn is
2 pi 2^-25 radians = 1.9e-7, sincospi 2 ulp), the two products and the sum three roundings more:
|err| <= 8e-7 A (|x_a| + |x_b|) before the last rounding, which adds half a step of the type, eps / 2 |y|.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def rotate64(x, pos, f, inter, amp, inverse):
    """x [T, H, d] float64 numpy -> (rotated, bound on |x_a| + |x_b| per element)."""
    r = 2 * f.size
    ang = pos.astype(np.float64)[:, None] * f[None] * (-1 if inverse else 1)
    c, s = (amp * np.cos(ang))[:, None], (amp * np.sin(ang))[:, None]
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if inter else (np.arange(r // 2), np.arange(r // 2, r))
    y, m = x.copy(), np.zeros_like(x)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    m[..., ia] = m[..., ib] = abs(amp) * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    return y, m


def close(got, want, mag, dtype):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    # positions far out: the reference's own angle is position * f rounded to 53 bits
    tol = 8e-7 * mag + torch.finfo(dtype).eps / 2 * np.abs(want) * (1 + 1e-6) + 1e-30
    bad = np.abs(g - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.abs(g - want).max():.3e}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 64, 64), (37, 5, 1, 128, 64), (300, 32, 8, 128, 128), (9, 3, 2, 80, 20),
                                           (5, 2, 1, 30, 14), (3, 2, 2, 64, 0), (130, 1, 1, 1024, 1024), (6, 1, 1, 7, 2)])
def test_rope(T, Hq, Hk, d, rot, inter, dtype):
    fa = need_gpu()
    g = torch.Generator().manual_seed(T + d)
    q, k = torch.randn(T, Hq, d, generator=g).to(dtype), torch.randn(T, Hk, d, generator=g).to(dtype)
    pos = torch.randint(-5, 2000000, (T,), generator=g, dtype=torch.int32)
    pos[0] = 2147483647 if T > 4 else 0
    f = fa.rope_frequencies(rot)[0] if rot else torch.zeros(0, dtype=torch.float64)
    for inverse, amp in ((False, 1.0), (True, 1.25)):
        qo, ko = fa.rope(q.cuda(), k.cuda(), f.cuda(), pos.cuda(), interleaved=inter, amplitude=amp, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            close(y, *rotate64(x.double().numpy(), pos.numpy(), f.numpy(), inter, amp, inverse), dtype)


def test_rope_views_batches_in_place_and_defaults():
    fa = need_gpu()
    B, N, Hq, Hk, d = 2, 33, 4, 2, 64
    x = torch.randn(B, N, (Hq + 2 * Hk) * d).to(torch.bfloat16)
    f = fa.rope_frequencies(32)[0]
    ref = [rotate64(t.reshape(B * N, -1, d).double().numpy(), np.tile(np.arange(N), B), f.numpy(), False, 1.0, False)
           for t in (x[..., :Hq * d].unflatten(-1, (Hq, d)), x[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d)))]
    for shift in (0, 3):                      # shift 3: views whose addresses take no 16-byte access
        buf = torch.zeros(B, N, (Hq + 2 * Hk) * d + shift, dtype=torch.bfloat16)
        buf[..., shift:] = x
        xb = buf.cuda()
        qv, kv = (xb[..., shift + a * d:shift + e * d].unflatten(-1, (e - a, d)) for a, e in ((0, Hq), (Hq, Hq + Hk)))
        for y, (w, m) in zip(fa.rope(qv, kv, f.cuda()), ref):
            close(y.reshape(B * N, -1, d), w, m, torch.bfloat16)
        before = xb.clone()
        fa.rope(qv, kv, f.cuda(), out_q=qv, out_k=kv)   # in place; v and the gap stay as they are
        for y, (w, m) in zip((qv, kv), ref):
            close(y.reshape(B * N, -1, d), w, m, torch.bfloat16)
        rest = shift + (Hq + Hk) * d
        assert torch.equal(xb[..., rest:], before[..., rest:]) and torch.equal(xb[..., :shift], before[..., :shift])
    # heads first: [B, H, N, d] seen as [B, N, H, d]; q alone
    qt = x[:1, :, :Hq * d].unflatten(-1, (Hq, d)).cuda().transpose(1, 2).contiguous().transpose(1, 2)
    close(fa.rope(qt, inv_freq=f.cuda())[0], ref[0][0][:N], ref[0][1][:N], torch.bfloat16)
    assert fa.rope(x.new_zeros(0, 4, 64).cuda(), inv_freq=f.cuda()).shape == (0, 4, 64)


def test_rope_inverse_is_the_gradient():
    """<R x, g> = <x, R^T g> in fp32, and the difference quotient of <R x, g> along a direction."""
    fa = need_gpu()
    x, g, e = (torch.randn(65, 3, 128).cuda() for _ in range(3))
    f = fa.rope_frequencies(96)[0].cuda()
    kw = dict(inv_freq=f, amplitude=1.3, interleaved=True)
    dx = fa.rope(g, inverse=True, **kw)
    val = lambda t: (fa.rope(t, **kw).double() * g.double()).sum()
    num = (val(x + 0.5 * e) - val(x - 0.5 * e)).item()
    # 25k products of size ~1.3 with relative errors of about 1e-6, signs at random: far below 25k * 1e-6 * 4
    assert abs(num - (dx.double() * e.double()).sum().item()) < 0.1


def test_rope_refusals():
    fa = need_gpu()
    f = fa.rope_frequencies(64)[0].cuda()
    q = torch.randn(4, 2, 64).to(torch.bfloat16).cuda()
    for bad in (lambda: fa.rope(q), lambda: fa.rope(q, inv_freq=f.float()), lambda: fa.rope(q.half(), inv_freq=f),
                lambda: fa.rope(q, q.float(), f), lambda: fa.rope(q, q[:3], f), lambda: fa.rope(q[:, :, ::2], inv_freq=f[:8]),
                lambda: fa.rope(q[..., :32], inv_freq=f), lambda: fa.rope(q.cpu(), inv_freq=f),
                lambda: fa.rope(q, inv_freq=f, positions=torch.zeros(4, dtype=torch.int64).cuda()),
                lambda: fa.rope(q, inv_freq=f, positions=torch.zeros(3, dtype=torch.int32).cuda()),
                lambda: fa.rope(q, inv_freq=f, out_q=q[:1].expand(4, 2, 64)),
                lambda: fa.rope(q, inv_freq=f, out_q=torch.empty(4, 2, 64, device="cuda")),
                lambda: fa.rope(q, inv_freq=f, out_k=q), lambda: fa.rope(q[0], inv_freq=f)):
        with pytest.raises((ValueError, TypeError)):
            bad()


@pytest.mark.parametrize("lens,chunks,page,Hq,Hkv,d,rot,inter", [
    ([1], [1], 16, 4, 4, 64, 64, False),
    ([5, 0, 40, 33], [1, 0, 1, 1], 16, 8, 2, 128, 64, True),
    ([70, 200, 17], [70, 3, 17], 32, 5, 1, 64, 32, False),
    ([9, 13], [4, 13], 3, 2, 2, 40, 20, False),
    ([130] * 300, [1] * 300, 128, 2, 1, 64, 64, True)])
def test_append(lens, chunks, page, Hq, Hkv, d, rot, inter):
    fa = need_gpu()
    B, T = len(lens), sum(chunks)
    pad = 3                                              # rows past the last chunk
    x = torch.randn(T + pad, (Hq + 2 * Hkv) * d).to(torch.bfloat16)
    q, k, v = (x[:, a * d:b * d].view(T + pad, b - a, d) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    per = [-(-n // page) for n in lens]
    maxp = max(per) + 1
    perm = torch.randperm(sum(per) + 2)
    table, o = torch.full((B, maxp), -7, dtype=torch.int32), 0
    for b, n in enumerate(per):
        table[b, :n], o = perm[o:o + n].int(), o + n
    kc, vc = (torch.randn(sum(per) + 2, page, Hkv, d).to(torch.bfloat16) for _ in range(2))
    f, cu = fa.rope_frequencies(rot)[0], np.concatenate([[0], np.cumsum(chunks)])
    t = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, chunks)])
    for pos in (None, torch.from_numpy(np.concatenate([t + 90000, np.zeros(pad)])).int()):
        kcg, vcg, xg = kc.cuda(), vc.cuda(), x.cuda()
        qg, kg, vg = (xg[:, a * d:b * d].view(T + pad, b - a, d) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        out = torch.full((T + pad, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        fa.rope_append_paged(qg, kg, vg, kcg, vcg, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             torch.from_numpy(cu).int().cuda(), f.cuda(), positions=None if pos is None else pos.cuda(),
                             interleaved=inter, amplitude=1.1, out=out)
        assert fa.debug_read_status() == 0
        p = t if pos is None else pos.numpy()[:T]
        close(out[:T], *rotate64(q[:T].double().numpy(), p, f.numpy(), inter, 1.1, False), torch.bfloat16)
        assert bool((out[T:] == 7).all())
        kr, km = rotate64(k[:T].double().numpy(), p, f.numpy(), inter, 1.1, False)
        want, mag, wv = kc.double().numpy(), np.zeros(kc.shape), vc.clone()
        for b in range(B):
            for r in range(cu[b], cu[b + 1]):
                pg, sl = table[b, t[r] // page], t[r] % page
                want[pg, sl], mag[pg, sl], wv[pg, sl] = kr[r], km[r], v[r]
        close(kcg, want, mag, torch.bfloat16)
        assert torch.equal(vcg.cpu(), wv)
    # without q
    kc2 = kc.cuda()
    assert fa.rope_append_paged(None, kg, vg, kc2, vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                torch.from_numpy(cu).int().cuda(), f.cuda(), positions=pos.cuda(), interleaved=inter,
                                amplitude=1.1) is None
    assert torch.equal(kc2, kcg)


def test_append_skips_bad_tables():
    """A page outside the pool, a chunk longer than its sequence and one past the table are skipped and recorded."""
    fa = need_gpu()
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    f = fa.rope_frequencies(64)[0].cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.rope_append_paged(None, k, k, kc, vc, i32([[9, 0], [1, 2], [3, 3], [3, 2]]), i32([3, 0, 33, 20]),
                         i32([0, 1, 2, 3, 4]), f)
    assert fa.debug_read_status() == fa.FATTN_ERR_DEVICE_CHECK
    assert bool((vc[2, 3] == 1).all()) and vc.sum() == 64


@pytest.mark.parametrize("inter", [False, True])
def test_rope_fp32_precision(inter):
    """Relative error of fp32 rotation, in the mean square. Rounding to p bits leaves an error of step / sqrt(12): an angle
    within a quarter of half a turn, 24 bits, pi 2^-26 0.76 / 3.46 = 1.0e-8 (0.76: the mean square of the steps over the
    binades below the quarter); sine and cosine 1.6e-8 each, 2.3e-8; the two products and their sum 3.4e-8 together:
    4.2e-8 in all. An angle held in 24 bits of the whole half turn alone adds four times the first, 4.1e-8."""
    fa = need_gpu()
    g = torch.Generator().manual_seed(1)
    T, d = 2000, 128
    x = torch.randn(T, 8, d, generator=g)
    pos = torch.randint(0, 2 ** 20, (T,), generator=g, dtype=torch.int32)
    f = fa.rope_frequencies(d)[0]
    for inverse in (False, True):
        y = fa.rope(x.cuda(), None, f.cuda(), pos.cuda(), interleaved=inter, inverse=inverse)
        want, _ = rotate64(x.double().numpy(), pos.numpy(), f.numpy(), inter, 1.0, inverse)
        err = np.sqrt(((y.double().cpu().numpy() - want) ** 2).sum() / (want ** 2).sum())
        assert err < 5.0e-8, err


def test_rope_quarter_turns():
    """Angles at and next to the quarter turns, of either sign, where sine and cosine swap: 2^k turns of a position."""
    fa = need_gpu()
    turns = torch.tensor([0.25, 0.5, 0.75, 1.0, 0.125, 0.375, 0.625, 0.875, 0.25 - 1e-9, 0.25 + 1e-9, 0.125 - 1e-9, 0.125 + 1e-9,
                          1e-9, 1 - 1e-9, 0.5 - 1e-9, 0.5 + 1e-9], dtype=torch.float64)
    f = turns * 2 * np.pi
    pos = torch.tensor([0, 1, -1, 2, 3, -3, 5, -7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    x = torch.randn(len(pos), 2, 32)
    for dtype in (torch.float32, torch.bfloat16):
        for inverse in (False, True):
            for inter in (False, True):
                xd = x.to(dtype)
                y = fa.rope(xd.cuda(), None, f.cuda(), pos.cuda(), interleaved=inter, inverse=inverse)
                near = pos.abs().long() < 100          # (far out the reference's product with 2 pi is off by more)
                near[-2:] = False
                want, mag = rotate64(xd.double().numpy(), pos.numpy(), f.numpy(), inter, 1.0, inverse)
                close(y[near.cuda()], want[near.numpy()], mag[near.numpy()], dtype)
                assert bool(torch.isfinite(y).all())
