"""The paged K/V cache beyond single calls: streams, graphs, inputs written just before, batches of many sequences and row
tiles, rows laid out as bf16 first, offsets past 32 bits, and the paged tests under device-side bounds checks."""
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
from test_gpu_paged import bits, compare, ints, lib, queries  # noqa: E402,F401

BF = torch.bfloat16


def call(lib, c, q, most, **kw):
    return lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, mask="causal", max_new=most, **c.scales, **kw)


MIXES = [(1, [900, 70, 333], [1, 1, 1]), (20, [900, 70, 333], [20, 3, 1]), (300, [900, 700, 333], [300, 3, 200])]


@pytest.mark.parametrize("most,lens,new", MIXES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("capacity", [0, 2000])  # items whole, and divided
def test_streams_and_graphs(lib, most, lens, new, int8, capacity):
    """Two calls at once on two streams, each with scratch of its own; captured calls replayed one after another."""
    cases = []
    for seed in (1, 2):
        c = pr.Cache(2, 16, lens, new, int8=int8, seed=seed, capacity=capacity).fill()
        cases.append((c, queries(c, 8, seed=seed)))
    want = [compare(lib, c, q, True) for c, q in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for s, (c, q) in zip(streams, cases):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(call(lib, c, q, most))
        torch.cuda.synchronize()
        assert all(torch.equal(a, z) for a, z in zip(want, got))
    for s in streams:  # a stream that is not the current one
        s.wait_stream(torch.cuda.current_stream())
    got = [call(lib, c, q, most, stream=s) for s, (c, q) in zip(streams, cases)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, z) for a, z in zip(want, got))
    graphs = []
    for c, q in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(lib, c, q, most)
        graphs.append((graph, out))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, out) for a, (_, out) in zip(want, graphs))


@pytest.mark.parametrize("int8", [False, True])
def test_a_captured_step_follows_lengths_tables_and_starts(lib, int8):
    """A decoding step captured once, for a batch and packed rows that are padded, and replayed as sequences grow, end and
    move to other pages: append, attention and reading back see what the tensors hold at each replay."""
    B, h, h_kv, page = 4, 4, 2, 16
    plans = [([17, 1, 30, 64], [1, 1, 1, 1]), ([18, 2, 31, 65], [1, 1, 1, 1]), ([90, 33, 0, 10], [5, 33, 0, 2]),
             ([90, 33, 128, 0], [0, 0, 20, 0])]
    N = 40
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    fixed = pr.Cache(h_kv, page, [128] * B, [0] * B, int8=int8, seed=4).fill()
    q, k, v = n(h, N, 64), n(h_kv, N, 64), n(h_kv, N, 64)
    starts, lens, out = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"), n(h, N, 64)
    table = fixed.page_table.clone()

    def step():
        lib.paged_cache_append(k, v, fixed.k_pages, fixed.v_pages, table, starts, lens, **fixed.scales)
        lib.sdpa_paged_forward(q, fixed.k_pages, fixed.v_pages, table, starts, lens, out, mask="causal", max_new=33, **fixed.scales)
        return lib.paged_cache_read(fixed.k_pages, fixed.v_pages, table, lens, rows=128, **fixed.scales)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        back = step()
    for i, (lengths, new) in enumerate(plans):
        c = pr.Cache(h_kv, page, lengths, new, int8=int8, seed=5 + i, capacity=128)
        c.page_table = fixed.page_table[torch.randperm(B, generator=torch.Generator().manual_seed(i)).to("cuda")].contiguous()
        c.k_pages, c.v_pages, c.k_scales, c.v_scales = fixed.k_pages, fixed.v_pages, fixed.k_scales, fixed.v_scales
        c.fill(new=False)
        for t in (k, v, q):
            t.copy_(n(*t.shape))
        for x, src in zip((k, v), c.packed_new()):
            x[:, :c.N] = src
        starts.copy_(c.row_starts)
        lens.copy_(c.seq_lens)
        table.copy_(c.page_table)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want, tol = pr.attend(q[:, :c.N], c, True)
        ref.check("o", out[:, :c.N], want, tol, 0)
        assert torch.all(out[:, c.N:] == 7)
        for b in range(B):
            for got, x in zip(back, c.cached(b)):
                assert torch.equal(got[b, :, :lengths[b]].double(), x) and torch.all(got[b, :, lengths[b]:] == 0)


@pytest.mark.parametrize("most,lens,new", MIXES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("capacity", [0, 2000])
def test_inputs_written_just_before(lib, most, lens, new, int8, capacity):
    """Everything a call reads is written right before it and destroyed right after it, eagerly and captured: launches may
    overlap the ends of the ones before them."""
    c = pr.Cache(2, 32, lens, new, int8=int8, seed=6, capacity=capacity).fill()
    q = queries(c, 8)
    want, (wk, wv) = call(lib, c, q, most), lib.paged_cache_read(*c.args, c.seq_lens, **c.scales)
    names = ["k_pages", "v_pages", "page_table", "row_starts", "seq_lens"] + (["k_scales", "v_scales"] if int8 else [])
    source = {n: getattr(c, n) for n in names}
    x, mq = {n: torch.empty_like(t) for n, t in source.items()}, torch.empty_like(q)

    def step():
        out = []
        for _ in range(3):
            for n, t in x.items():
                t.copy_(source[n])
                setattr(c, n, t)
            mq.copy_(q)
            out.append((call(lib, c, mq, most), *lib.paged_cache_read(*c.args, c.seq_lens, **c.scales)))
            for n, t in x.items():
                t.fill_(1 if t.dtype is torch.uint8 else 0)
            mq.fill_(float("nan"))
        return out

    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o, k, v in eager + captured:
        assert torch.equal(o, want) and torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.parametrize("int8", [False, True])
def test_append_then_attend_at_once(lib, int8):
    """The attention launched right behind the append that writes the rows it reads, over and over."""
    c = pr.Cache(4, 16, [400] * 6, [1] * 6, int8=int8, seed=7).fill()
    k, v = c.packed_new()
    q = queries(c, 8)
    want = call(lib, c, q, 1)
    for _ in range(20):
        for b in range(c.B):  # the new row's place forgotten
            pg, at = c.page_table[b, 399 // 16].long(), 399 % 16
            c.k_pages[pg, :, at] = 0
            c.v_pages[pg, :, at] = 0
        lib.paged_cache_append(k, v, *c.args, c.row_starts, c.seq_lens, **c.scales)
        assert torch.equal(call(lib, c, q, 1), want)


# (h, h_kv, page, lengths, new): more sequences than a block has threads, empty ones among them; more pieces a CTA than its
# table holds; shares that end inside every kind of item
MANY = [(4, 4, 16, [20 + 7 * (i % 5) for i in range(300)], [1 if i % 3 else 0 for i in range(300)]),
        (8, 4, 16, [37 + i % 90 for i in range(500)], [1 + i % 2 for i in range(500)]),
        (64, 64, 16, [40 + i % 60 for i in range(150)], [40 - i % 3 for i in range(150)]),
        (8, 1, 32, [300 + i for i in range(140)], [3 if i % 20 else 40 for i in range(140)])]


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("int8", [False, True])
def test_many_sequences(lib, shape, int8):
    h, *rest = shape
    c = pr.Cache(*rest, int8=int8, seed=8).fill()
    compare(lib, c, queries(c, h, 2.0), True)


# (h, h_kv, page, lengths, new) in tables of 2,000 rows, whose items are divided: so short that workers' shares end before the
# first key of an item, or hold one piece's last keys and another's beginning
SHORT = [(1, 1, 16, [1], [1]), (4, 2, 16, [17, 1, 0, 33, 64], [1, 1, 0, 1, 1]), (8, 8, 32, [1 + i % 40 for i in range(40)], [1] * 40),
         (16, 16, 16, [5 + i for i in range(130)], [1 + i % 3 for i in range(130)]), (8, 1, 64, [500, 3, 900, 64], [1, 1, 2, 0]),
         (12, 4, 48, [1999, 1, 1, 1500], [1, 1, 1, 4])]


@pytest.mark.parametrize("shape", SHORT)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("most", [None, 40])
def test_short_items_that_are_divided(lib, shape, int8, most):
    h, *rest = shape
    c = pr.Cache(*rest, int8=int8, seed=12, capacity=2000).fill()
    out = compare(lib, c, queries(c, h, 2.0), True, max_new=max(c.new) if most is None else most)
    again = compare(lib, c, queries(c, h, 2.0), True, max_new=max(c.new) if most is None else most)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


# (h, h_kv, page, lengths, new): int8 rows, and pages of 16, 48 and 32 rows, that are laid out as bf16 first, some sequences
# of a batch among others that are not
WIDE = [(8, 2, 16, [700], [200]), (4, 1, 48, [300, 1000, 50, 129], [130, 200, 1, 129]), (16, 2, 32, [520, 2, 900], [513, 1, 7]),
        (2, 2, 64, [1500, 1300], [600, 900]), (6, 2, 16, [130, 640, 256, 7], [130, 0, 200, 7])]


@pytest.mark.parametrize("shape", WIDE)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_laid_out_first(lib, shape, int8, causal):
    h, *rest = shape
    c = pr.Cache(*rest, int8=int8, seed=9).fill()
    compare(lib, c, queries(c, h, 3.0), causal)
    # pages that are not there, in the first, a middle and the last tile
    gone = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in c.lens]
    for b, n in enumerate(c.lens):
        for i in {0, n // 2 // c.page, (n - 1) // c.page} if n else ():
            if i != (n - 1) // c.page or n > 2 * c.page:
                c.page_table[b, i] = -1
                gone[b][i * c.page:(i + 1) * c.page] = True
    compare(lib, c, queries(c, h, 3.0), causal, gone)


@pytest.mark.parametrize("new", [1, 33, 300])
@pytest.mark.parametrize("int8", [False, True])
def test_offsets_past_32_bits(lib, new, int8):
    """Pages, queries and outputs further apart than 32 bits of elements, let alone bytes."""
    c = pr.Cache(2, 16, [400, 310], [new, new], int8=int8, seed=10).fill()
    q = queries(c, 4)
    want = compare(lib, c, q, True)
    few = pr.Cache(2, 256, [400, 310], [new, new], int8=int8, seed=10)
    dtype = torch.int8 if int8 else BF
    stride, size = (1 << 31) + 64, 2 * 256 * 64
    pool = torch.zeros(3 * stride + 2 * size, dtype=dtype, device="cuda")
    few.pages = 4
    few.page_table = ints(3, 0, 1, 2).reshape(2, 2)
    few.k_pages = torch.as_strided(pool, (4, 2, 256, 64), (stride, 256 * 64, 64, 1), 0)
    few.v_pages = torch.as_strided(pool, (4, 2, 256, 64), (stride, 256 * 64, 64, 1), size)
    if int8:
        few.k_scales, few.v_scales = (torch.full((4, 2, 256), 255, dtype=torch.uint8, device="cuda") for _ in "kv")
    few.rows = c.rows
    few.fill(new=False)
    k, v = c.packed_new()
    lib.paged_cache_append(k, v, *few.args, few.row_starts, few.seq_lens, **few.scales)
    for x, z in zip(lib.paged_cache_read(*few.args, few.seq_lens, rows=400, **few.scales),
                    lib.paged_cache_read(*c.args, c.seq_lens, rows=400, **c.scales)):
        assert torch.equal(x, z)
    got = compare(lib, few, q, True)
    far = torch.as_strided(torch.zeros(3 * stride + c.N * 64, dtype=BF, device="cuda"), (4, c.N, 64), (stride, 64, 1))
    out = torch.as_strided(torch.zeros(3 * stride + c.N * 64, dtype=BF, device="cuda"), (4, c.N, 64), (stride, 64, 1))
    far.copy_(q)
    lib.sdpa_paged_forward(far, *few.args, few.row_starts, few.seq_lens, out, mask="causal", max_new=new, **few.scales)
    assert torch.equal(out, got)
    assert (got.double() - want.double()).norm() <= 2 * pr.U * want.double().norm()


def test_long_sequences(lib):
    """Positions past 2^17 and lengths that divide over every worker; the exact weights of the last tokens."""
    for int8, new in ((False, 1), (True, 3), (True, 40)):
        c = pr.Cache(1, 64, [200_001], [new], int8=int8, seed=11).fill()
        compare(lib, c, queries(c, 4, 4.0), True)


def test_refusals_on_the_device(lib):
    c = pr.Cache(2, 16, [40, 30], [3, 1], capacity=2000).fill()
    q = queries(c, 4)
    with pytest.raises(ValueError):  # not contiguous in the last dimension
        call(lib, c, torch.cat((q, q), 2)[:, :, ::2], 3)
    with pytest.raises(lib.MhaError):  # heads on top of one another
        call(lib, c, q[:1].expand(4, -1, -1), 3)
    with pytest.raises(lib.MhaError):  # a row's 16 bytes divided
        call(lib, c, torch.as_strided(torch.zeros(9000, dtype=BF, device="cuda"), (4, 4, 64), (68 * 4, 68, 1)), 3)
    with pytest.raises(lib.MhaError):
        call(lib, c, q, 3, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.MhaError):
        call(lib, c, queries(c, 3), 3)
    pool = torch.zeros(20, 16, 2, 64, dtype=BF, device="cuda").transpose(1, 2)
    with pytest.raises(ValueError):  # pages row by row
        lib.paged_cache_read(pool, pool, c.page_table, c.seq_lens)
    with pytest.raises(ValueError):
        lib.sdpa_paged_forward(q, *c.args, None, c.seq_lens)
    with pytest.raises(ValueError):
        lib.paged_cache_append(q[:2].cpu(), q[:2], *c.args, c.row_starts, c.seq_lens)


def test_paged_cases_pass_with_bounds_checks():
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
         os.path.join("tests", "test_gpu_paged.py"), os.path.join("tests", "test_gpu_paged_more.py"),
         "-k", "not bounds_checks and not past_32_bits"],
        cwd=ROOT, env=dict(os.environ, MHA_LIBRARY=_checked_library()), capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert int(re.search(r"(\d+) passed", r.stdout).group(1)) >= 230, r.stdout[-2000:]
