"""The limits that include/mha.h states for sdpa_paged_forward, on both sides of each, without a GPU: sizes whose work 32 bits
do not number, and calls that need no workspace.  (No call here gets past its checks.)"""
import ctypes

import pytest

from test_paged_host import attend, cache, nat  # noqa: F401

LINE = (1 << 31) - (1 << 14)
H_KV = 64


def make(nat, int8, **kw):
    return cache(nat, dtype=nat.MHA_INT8 if int8 else nat.MHA_BF16, k_scales=1 << 20 if int8 else None,
                 v_scales=1 << 20 if int8 else None, **kw)


def both_refuse(nat, c, h, N, most):
    """Whether the call is refused for its size; the query and the call have to agree."""
    need = nat.lib.sdpa_paged_workspace_bytes(ctypes.addressof(c), h, N, most)
    got = attend(nat, c, h=h, N=N, most=most, qh=64 * N, oh=64 * N, ws=None)
    assert (need, got) == (0, nat.MHA_ERR_UNSUPPORTED) or (need > 0 and got == nat.MHA_ERR_WORKSPACE), (need, got)
    return need == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("most,times", [(1, 1), (5, 1), (40, None)])
@pytest.mark.parametrize("cap", [1 << 20, (1 << 20) + 16])
def test_sequences_that_32_bits_number(nat, int8, most, times, cap):
    """B h_kv (c / 16 + 17), with int8 c / 32: past 16 (int8 32) rows of a K/V head twice (four times)."""
    times = times or (4 if int8 else 2)
    units = cap // (32 if int8 else 16) + 17
    last = (LINE - 1) // (H_KV * times * units)
    sizes = dict(h_kv=H_KV, page_stride=H_KV * 16 * 64, max_pages=cap // 16)
    for B, refused in ((last, False), (last + 1, True), (1, False), (65535, True)):
        assert both_refuse(nat, make(nat, int8, B=B, **sizes), H_KV, 600, most) == refused, B


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("g", [1, 3, 128])
def test_row_tiles_that_32_bits_number(nat, int8, g):
    """(ceil(N / floor(128 / g)) + B) h_kv (c / 128 + 8)."""
    h_kv, cap, B = 4, 1 << 22, 3
    c = make(nat, int8, h_kv=h_kv, page_stride=h_kv * 16 * 64, max_pages=cap // 16, B=B)
    tiles = (LINE - 1) // (h_kv * (cap // 128 + 8)) - B
    last = tiles * (128 // g)
    assert last * g * h_kv < 1 << 30
    for N, refused in ((last, False), (last + 1, True)):
        assert both_refuse(nat, c, g * h_kv, N, N) == refused, N


def test_heads_of_a_group_count_once(nat):
    """With more query heads a K/V head than there are few rows no sequence is taken so: they are no reason to refuse."""
    cap = 1 << 20
    last = (LINE - 1) // (2 * (cap // 16 + 17))
    c = make(nat, False, h_kv=1, page_stride=16 * 64, max_pages=cap // 16, B=last)
    assert not both_refuse(nat, c, 128, 600, 1)


@pytest.mark.parametrize("int8,rows,items", [(False, 1, 608), (False, 8, 608), (False, 9, 456), (False, 16, 456), (True, 8, 608),
                                             (True, 16, 456), (True, 17, 304), (True, 32, 304)])
def test_calls_without_a_workspace(nat, int8, rows, items):
    def need(B, rows=rows, max_pages=64):
        c = make(nat, int8, B=B, h_kv=4, max_pages=max_pages)
        return nat.lib.sdpa_paged_workspace_bytes(ctypes.addressof(c), 4, 10 ** 5, rows)

    assert need(items // 4) == 0 < need(items // 4 + 1)
    assert need(1, max_pages=65) > 0
    assert need(1, rows=33 if int8 else 17) > 0
