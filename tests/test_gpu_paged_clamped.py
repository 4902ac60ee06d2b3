"""Attention over a paged cache with lengths and starts out of range on the device: as with the clamped ones, and nothing past
the packed rows is touched.  And what row-tile kernels make of long chunks straight from their pages, where laying the rows out
as bf16 first would take too much."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402
import scored_reference as ref  # noqa: E402
from test_gpu_bounds_checked import ROOT, _checked_library  # noqa: E402
from test_gpu_paged import BF, compare, ints, lib, queries  # noqa: E402,F401

GUARD = 40  # rows behind the packed ones


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [112, 2000])   # items whole, and divided
@pytest.mark.parametrize("heads,last", [((2, 2), 4), ((4, 2), 60), ((4, 2), 300)])  # few rows, row tiles, rows laid out first
def test_lengths_and_starts_out_of_range(lib, int8, causal, cap, heads, last):
    h, h_kv = heads
    N = 8 + last
    c = pr.Cache(h_kv, 16, [cap] * 4, [0] * 4, int8=int8, seed=51).fill()
    assert c.max_pages * 16 == cap
    q = torch.randn(h, N + GUARD, 64, generator=c.g, device="cuda").to(BF)
    q[:, N:] = float("nan")

    def call(starts, lens):
        out = torch.full((h, N + GUARD, 64), 5.0, dtype=BF, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.sdpa_paged_forward(q[:, :N], *c.args, ints(*starts), ints(*lens), out[:, :N], status=status,
                               mask="causal" if causal else "none", **c.scales)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and torch.all(out[:, N:] == 5)
        return out[:, :N]

    got = call((-4, 3, 3, 8, 9000), (-1, 50, 1 << 30, cap + 1))
    assert torch.all(got[:, :3] == 0)
    assert torch.equal(got, call((0, 3, 3, 8, N), (0, 50, cap, cap)))
    # the same from the definition
    c.lens, c.new, c.starts, c.N = [0, 50, cap, cap], [3, 0, 5, last], [0, 3, 3, 8, N], N
    c.rows = [tuple(x[:, :n] for x in rows) for rows, n in zip(c.rows, c.lens)]
    want, tol = pr.attend(q[:, :N], c, causal)
    ref.check("o", got, want, tol, 0)
    # no sequence has rows, or none of the packed ones
    assert torch.all(call((0, 3, 3, 8, N), (0, -5, -(1 << 31), 0)) == torch.tensor([0.0], device="cuda", dtype=BF))
    assert torch.all(call((N, 1 << 30, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1), (cap,) * 4) == 5)
    assert torch.all(call((-9, -7, -7, -1, 0), (cap,) * 4) == 5)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30])
def test_scales_report_no_status(lib, int8, scale):
    c = pr.Cache(1, 16, [90, 400], [1, 150], int8=int8, seed=12).fill()
    q, status = queries(c, 2), torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, scale=scale, mask="causal", status=status, **c.scales)
    torch.cuda.synchronize()
    assert int(status.item()) == 0


# (h, h_kv, page, lengths, new, max_new, table rows): chunks of several row tiles; short sequences with more pieces a CTA than
# its table holds; each among sequences of a few rows
STRAIGHT = [(4, 2, 64, [1500, 700, 90], [600, 300, 1], 600, 1 << 22), (8, 2, 16, [900, 2, 1300], [513, 1, 131], 513, 1 << 22),
            (6, 2, 48, [640, 1000], [640, 7], 640, 1 << 23), (4, 4, 32, [2300], [2100], 2100, 1 << 23),
            (64, 64, 16, [40 + i % 60 for i in range(150)], [40 - i % 3 for i in range(150)], 600, 2000)]


@pytest.mark.parametrize("shape", STRAIGHT)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_long_chunks_straight_from_their_pages(lib, shape, int8, causal):
    h, h_kv, page, lens, new, most, table = shape
    c = pr.Cache(h_kv, page, lens, new, int8=int8, seed=52).fill()
    q = queries(c, h, 2.0)

    def need():
        packed = lib._paged_cache(torch, *c.args, c.row_starts, c.seq_lens, c.k_scales, c.v_scales)[0]
        return lib.lib.sdpa_paged_workspace_bytes(packed, h, c.N, most)

    trimmed, narrow = compare(lib, c, q, causal, max_new=most), need()
    wide = torch.full((c.B, table // page + 1), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.max_pages] = c.page_table
    c.page_table = wide
    # no room for the rows of the whole table, of at least one sequence
    assert need() < 2 * h_kv * table * 128 and need() <= narrow + (1 << 22)
    got = compare(lib, c, q, causal, max_new=most)
    assert (got.double() - trimmed.double()).norm() <= 2 * pr.U * trimmed.double().norm()
    assert torch.equal(got, compare(lib, c, q, causal, max_new=most))


def test_cases_pass_with_bounds_checks():
    here = ["test_gpu_paged_clamped.py", "test_gpu_paged_small_values.py", "test_gpu_scored_windows.py", "test_gpu_paged_runs.py",
            "test_gpu_forward_runs.py"]
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *(os.path.join("tests", n) for n in here),
         "-k", "not bounds_checks and not shape4"],
        cwd=ROOT, env=dict(os.environ, MHA_LIBRARY=_checked_library()), capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert int(re.search(r"(\d+) passed", r.stdout).group(1)) >= 400, r.stdout[-2000:]
