"""The 8-bit block-scaled cache without a GPU: sizes near and beyond the ends of int32 are refused."""
import pytest

from compressed_domain_attention_tq_b200 import _lib
from test_boundary_host import lib  # noqa: F401
from test_q8_host import INVALID, call


@pytest.mark.parametrize("what", ["append", "read"])
@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 2])
def test_tokens_near_the_last_int32(lib, what, n):  # noqa: F811
    assert call(lib, what, n=n, B=1, Hkv=1, block=128) == INVALID


@pytest.mark.parametrize("at", range(6))
def test_workspace_of_sizes_beyond_int32_is_zero(lib, at):  # noqa: F811
    """Not what the sizes' low 32 bits would need."""
    args = [1, 8, 8, 128, 1, 100]
    assert _lib.sdpa_q8_workspace_bytes(*args) > 0
    args[at] += 1 << 32
    assert _lib.sdpa_q8_workspace_bytes(*args) == 0
