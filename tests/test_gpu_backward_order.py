"""The backward's pipeline with late roles: every launch finds its code and inputs out of L2, so the
roles of a block start and refill at different times."""
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _cold(n=64 << 20):
    torch.empty(n, device="cuda").fill_(0.0)      # 256 MB: more than L2


@pytest.mark.parametrize("d", [64, 128])
def test_cold_launches_do_not_stop(d):
    """dS of two tiles in flight: a late issuer must not miss the first one's barrier phase. No wait runs out and
    repeated launches agree bit for bit."""
    fa = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(d)
    r = lambda h: (torch.randn(2, 8192, h, d, generator=g, device="cuda") * 2).to(torch.bfloat16)
    q, k, v, do = r(32), r(8), r(8), r(32)
    for name, extra in (("plain", {}), ("shaped", {}), ("shaped", dict(window=4096)),
                        ("shaped", dict(slopes=torch.rand(32, device="cuda")))):
        fwd, bwd = (fa.fwd, fa.bwd) if name == "plain" else (fa.fwd_shaped, fa.bwd_shaped)
        o, lse = fwd(q, k, v, causal=True, **extra)
        first = None
        for _ in range(3):
            _cold()
            got = bwd(q, k, v, o, lse, do, causal=True, **extra)
            assert fa.debug_read_status() == 0, (name, extra)
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got))
