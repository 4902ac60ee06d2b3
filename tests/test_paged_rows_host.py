"""Packed rows that 32 bits number."""
import pytest

from test_paged_host import append, cache, nat  # noqa: F401


@pytest.mark.parametrize("N", [1 << 30, (1 << 31) - 1])
def test_append_refuses_rows_past_its_grid(nat, N):
    """Token numbers round up to a block's 32: close to 2^31 they would not be 32-bit numbers."""
    assert append(nat, cache(nat), N=N, kh=64 << 31, vh=64 << 31) == nat.MHA_ERR_UNSUPPORTED
