"""Packed rows' starts at the ends of their type: cut to the packed rows like any other."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402
from test_gpu_paged import BF, bits, ints, lib  # noqa: E402,F401

LEAST, MOST = -(1 << 31), (1 << 31) - 1


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("last", [1, 60])
def test_the_least_and_the_largest_start(lib, int8, last):
    N = 3 + last
    q = torch.randn(2, N, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    caches = [pr.Cache(2, 16, [112] * 4, [0] * 4, int8=int8, seed=53, capacity=300).fill() for _ in range(2)]
    outs = []
    # the first two sequences have no rows, the third rows 0 .. 2, the last the others
    for c, starts in zip(caches, ((2, LEAST, LEAST, 3, MOST), (0, 0, 0, 3, N))):
        lib.paged_cache_append(q, q, *c.args, ints(*starts), c.seq_lens, **c.scales)
        outs.append(lib.sdpa_paged_forward(q, *c.args, ints(*starts), c.seq_lens, mask="causal", **c.scales))
    assert torch.equal(*outs) and bool(torch.isfinite(outs[0]).all())
    for name in ("k_pages", "v_pages"):
        assert torch.equal(bits(getattr(caches[0], name)), bits(getattr(caches[1], name)))
