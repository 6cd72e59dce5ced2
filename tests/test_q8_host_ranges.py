"""The 8-bit block-scaled cache without a GPU: sizes near and beyond the ends of int32 are refused."""
import pytest

from compressed_domain_attention_tq_b200 import _lib
from test_boundary_host import lib  # noqa: F401
from test_q8_host import INVALID, call


@pytest.mark.parametrize("what", ["append", "read"])
@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 2])
def test_tokens_near_the_last_int32(lib, what, n):  # noqa: F811
    assert call(lib, what, n=n, B=1, Hkv=1, block=128) == INVALID
