"""Chunks over pages of 32 rows: laid out as bf16 first where the table has 8,192 rows or more, else straight from the pages."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402
from test_gpu_paged import compare, lib, queries  # noqa: E402,F401


@pytest.mark.parametrize("rows,first", [(8160, False), (8192, True)])
@pytest.mark.parametrize("page", [32, 96])
@pytest.mark.parametrize("causal", [True, False])
def test_both_sides_of_the_rule(lib, rows, first, page, causal):
    rows += page - 32  # (the same side of the rule)
    c = pr.Cache(2, page, [520, 2, 900], [513, 1, 7], seed=9, capacity=rows // page * page).fill()
    q = queries(c, 16, 3.0)

    def need(most):
        packed = lib._paged_cache(torch, *c.args, c.row_starts, c.seq_lens, None, None)[0]
        return lib.lib.sdpa_paged_workspace_bytes(packed, 16, c.N, most)

    room = 3 * 2 * (rows // 128) * 128 * 256  # of three tables
    if page == 32:
        assert (need(513) - need(200) >= room) == first
    o = compare(lib, c, q, causal)
    assert torch.equal(o, compare(lib, c, q, causal))
    # a page that is not there
    gone = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in c.lens]
    for b, i in ((0, 1), (2, 900 // page - 1)):
        c.page_table[b, i] = -1
        gone[b][i * page:(i + 1) * page] = True
    compare(lib, c, q, causal, gone)
