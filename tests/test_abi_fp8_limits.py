"""Limits of the chunks over the 8-bit cache, without a GPU: what only the bf16 copy cannot do is refused to it alone, and
before anything is launched. (A call that passes the limits is stopped by its missing workspace.)"""
import pytest

from exact_tiled_attention_fattn_gb300 import build as fbuild
from exact_tiled_attention_fattn_gb300 import fattn as F
from tests.test_abi_fp8_cache import _chunk

WORKSPACE, UNSUPPORTED = F.FATTN_ERR_WORKSPACE, F.FATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return F.load_library()


def test_tables_past_the_copy(lib):
    """Two tables of 2^26 pages of 16 tokens: more slots than the copy may have, no matter for streamed rows."""
    few, many = dict(mq=5, T=10), dict(mq=200, T=400)
    wide = dict(maxp=1 << 26, ws=None)
    assert _chunk(lib, **few, **wide) == WORKSPACE and _chunk(lib, **many, **wide) == UNSUPPORTED
    assert _chunk(lib, **many, maxp=(1 << 26) - 1, ws=None) == WORKSPACE           # (2^31 - 16 slots with one more page)
    assert _chunk(lib, **few, maxp=(1 << 27) - 65, ws=None) == WORKSPACE           # 2^31 - 1040 tokens
    # 2 x 32 groups of that many steps are more than an int
    assert _chunk(lib, **few, Hq=64, Hkv=32, maxp=(1 << 27) - 65, ws=None) == UNSUPPORTED


def test_many_sequences(lib):
    B = 70000
    assert _chunk(lib, B=B, T=B, mq=2, S=1, ws=None) == _chunk(lib, B=B, T=B, mq=2, S=4, ws=None) == WORKSPACE
    assert _chunk(lib, B=B, T=B + 300, mq=200, S=1, ws=None) == WORKSPACE
    assert _chunk(lib, B=B, T=B + 300, mq=200, S=2, ws=None) == UNSUPPORTED        # the joining launch's grid


def test_items_and_rows(lib):
    assert _chunk(lib, T=1 << 28, mq=1 << 28, S=2, ws=None) == UNSUPPORTED         # 2^28 rows of 4 heads in two pieces
    assert _chunk(lib, T=1 << 20, mq=1 << 30, S=3, ws=None) == UNSUPPORTED         # longest chunk times heads
