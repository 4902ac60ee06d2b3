"""The paged K/V cache (paged_cache_append, paged_cache_read) and attention over it (sdpa_paged_forward) against their
definitions in fp64."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402
import scored_reference as ref  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    import transformer_scaled_dot_softmax_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def bits(x):
    return x.view(torch.int16) if x.dtype is BF else x


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def token_major(x):
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def queries(c, h, gain=1.0, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(h, c.N, 64, generator=g, device="cuda") * gain).to(BF)


def compare(lib, c, q, causal, gone=None, **kw):
    """One call into an output of NaN, checked; what it wrote."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kw.pop("out", None)
    out = torch.full_like(q, float("nan")) if out is None else out
    lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, out, mask="causal" if causal else "none", status=status,
                           **{"max_new": max(c.new + [0]), **c.scales, **kw})
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want, tol = pr.attend(q, c, causal, kw.get("scale") or 0.125, gone)
    ref.check("o", out[:, :c.N], want, tol, 2, q.shape[0] * c.N)
    return out


# ------------------------------------------------------------------------------------------------------ the cache
# (h_kv, page rows, lengths, new rows): whole prompts, single tokens, chunks that begin and end inside pages, nothing new
CACHES = [(1, 16, [1], [1]), (3, 16, [5, 16, 17, 40], [5, 1, 17, 0]), (2, 48, [100, 200, 47], [30, 1, 47]),
          (16, 64, [64, 65, 1000], [64, 1, 333]), (5, 128, [300, 0, 129], [299, 0, 2]), (8, 256, [700], [700])]


@pytest.mark.parametrize("shape", CACHES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("by_token", [False, True])
def test_append_writes_the_new_rows_and_nothing_else(lib, shape, int8, by_token):
    c, want = (pr.Cache(*shape, int8=int8, seed=3, capacity=400) for _ in range(2))
    c.fill(new=False)
    want.fill()
    k, v = c.packed_new()
    if by_token:
        k, v = token_major(k), token_major(v)
    r = lib.paged_cache_append(k, v, *c.args, c.row_starts, c.seq_lens, **c.scales)
    assert r[0] is c.k_pages and r[1] is c.v_pages
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        if getattr(c, name) is not None:
            assert torch.equal(bits(getattr(c, name)), bits(getattr(want, name))), name


@pytest.mark.parametrize("shape", CACHES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows", [None, 1, 33, 1024])
def test_read_returns_the_rows_and_zeros_behind_them(lib, shape, int8, rows):
    c = pr.Cache(*shape, int8=int8, seed=4, capacity=300).fill()
    k, v = lib.paged_cache_read(*c.args, c.seq_lens, rows=rows, **c.scales)
    T = c.max_pages * c.page if rows is None else rows
    assert k.shape == v.shape == (c.B, c.h_kv, T, 64)
    for b in range(c.B):
        n = min(c.lens[b], T)
        for got, x in zip((k, v), c.cached(b)):
            assert torch.equal(got[b, :, :n].double(), x[:, :n]) and torch.all(got[b, :, n:].view(torch.int16) == 0)


def extreme_rows():
    """Rows whose exponent, rounding or range is at an edge."""
    x = torch.zeros(24, 64, dtype=torch.float64)
    ramp = torch.arange(64, dtype=torch.float64)
    x[1, 5] = 2.0 ** -133                      # the least bf16 number
    x[2] = (ramp - 32) * 2.0 ** -130           # subnormal and normal numbers
    x[3] = ramp * 2.0 ** 120                   # near the largest numbers
    x[4, 0], x[4, 1] = 127.0, 63.5             # 127 steps exactly, a half step to even
    x[5, 0], x[5, 1] = 127.5, 126.5            # the mantissa past 127 / 128: a wider step
    x[6, 0], x[6, 1:4] = 127.0, torch.tensor([0.5, 1.5, 2.5], dtype=torch.float64)
    x[7, 0], x[7, 1:4] = 127.0, torch.tensor([-0.5, -1.5, -2.5], dtype=torch.float64)
    x[8] = -1.0
    x[9, 63] = float("nan")
    x[10, 0] = float("inf")
    x[11, 8] = float("-inf")
    x[12] = torch.finfo(BF).max
    x[13] = -torch.finfo(BF).max
    x[14, 0], x[14, 1] = 1.0, 2.0 ** -60       # far apart
    x[15] = 2.0 ** -126
    x[16] = 127 * 2.0 ** -126
    x[17] = 128 * 2.0 ** -126
    x[18, 0] = 254.0
    x[19, 0] = 255.0
    x[20, 0] = 256.0
    x[21, 0] = -127.5
    x[22] = ramp
    x[23] = -ramp / 63
    return x.to(BF)


def test_rows_at_the_edges_of_the_eight_bit_form(lib):
    x = extreme_rows().cuda()[None]
    c = pr.Cache(1, 16, [24], [24], int8=True)
    c.rows = [(x, x.flip(1))]
    lib.paged_cache_append(x, x.flip(1).contiguous(), *c.args, c.row_starts, c.seq_lens, **c.scales)
    want = pr.Cache(1, 16, [24], [24], int8=True)
    want.rows = c.rows
    want.fill()
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        assert torch.equal(getattr(c, name), getattr(want, name)), name
    k, v = lib.paged_cache_read(*c.args, c.seq_lens, rows=24, **c.scales)
    for got, kept, rows in zip((k[0], v[0]), c.cached(0), (x, x.flip(1))):
        assert torch.equal(torch.isnan(got), torch.isnan(kept))
        fine = ~torch.isnan(kept)
        assert torch.equal(got.double()[fine], kept[fine])
        # off by at most half a step, and by less than 1/127 of the row's largest; by 3/4 of a step of 2^122 at the
        # largest numbers
        rows = rows.double()
        top, off = rows.abs().amax(-1), (kept - rows).abs().amax(-1)
        last = top == torch.finfo(BF).max
        ok = torch.isfinite(top) & (top >= 127 * 2.0 ** -126) & ~last
        assert torch.all(off[ok] * 127 < top[ok]) and torch.all(off[last] == 0.75 * 2.0 ** 122)


@pytest.mark.parametrize("int8", [False, True])
def test_rows_without_a_place_are_dropped(lib, int8):
    """Positions below 0, pages that are not there, packed rows of no sequence, starts and lengths out of range."""
    c = pr.Cache(2, 16, [40, 30, 20, 33], [20, 8, 20, 5], int8=int8, seed=6)
    before = [t.clone() for t in (c.k_pages, c.v_pages)]
    k, v = c.packed_new()
    pad = torch.full((2, 3, 64), 7.0, dtype=BF, device="cuda")
    k, v = torch.cat((pad, k, pad), 1), torch.cat((pad, v, pad), 1)
    starts = c.row_starts + 3
    table = c.page_table.clone()
    table[0, 2] = -1               # rows 32 .. 39 of sequence 0
    table[1, 1] = c.pages          # rows 16 .. 29 of sequence 1
    lens = c.seq_lens.clone()
    lens[2] = 12                   # its first 8 new rows lie before the sequence
    lib.paged_cache_append(k, v, c.k_pages, c.v_pages, table, starts, lens, **c.scales)
    w = pr.Cache(2, 16, [40, 30, 20, 33], [20, 8, 20, 5], int8=int8, seed=6)
    w.put(0, 20, 32)
    w.rows[2] = tuple(x[:, 8:] for x in w.rows[2])
    w.put(2, 0, 12)
    w.put(3, 28, 33)
    for name in ("k_pages", "v_pages"):
        assert torch.equal(bits(getattr(c, name)), bits(getattr(w, name))), name
    # nothing at all: no length, or starts that leave the packed rows
    for args in ((starts, torch.zeros_like(lens)), (starts + 1000, c.seq_lens), (starts * 0 - 5, c.seq_lens)):
        d = pr.Cache(2, 16, [40, 30, 20, 33], [20, 8, 20, 5], int8=int8, seed=6)
        lib.paged_cache_append(k, v, d.k_pages, d.v_pages, table, *args, **d.scales)
        assert all(torch.equal(bits(a), bits(z)) for a, z in zip(before, (d.k_pages, d.v_pages)))


@pytest.mark.parametrize("int8", [False, True])
def test_pages_that_are_not_there_read_as_zeros(lib, int8):
    c = pr.Cache(2, 32, [100, 64], [0, 0], int8=int8, seed=7).fill()
    table = c.page_table.clone()
    table[0, 1], table[1, 0] = -7, 1 << 30
    k, v = lib.paged_cache_read(c.k_pages, c.v_pages, table, ints(100, 1 << 20), rows=128, **c.scales)
    for got, i in ((k, 0), (v, 1)):
        want = torch.zeros(2, 2, 128, 64, dtype=torch.float64, device="cuda")
        want[0, :, :100], want[1, :, :64] = c.cached(0)[i], c.cached(1)[i]
        want[0, :, 32:64] = 0
        want[1, :, :32] = 0
        assert torch.equal(got[:, :, :64].double(), want[:, :, :64])
        assert torch.equal(got[0].double(), want[0])


# ---------------------------------------------------------------------------------------------------- attention
# (h, h_kv, page rows, lengths, new rows): single tokens, drafted tokens, every size of the stacked rows around 8, 16,
# 32, 64 and 128, chunks, prompts, all of them mixed, sequences without new tokens or without rows
SHAPES = [(1, 1, 16, [1], [1]), (4, 2, 16, [5, 16, 17, 100], [1, 1, 1, 1]), (8, 1, 16, [333, 15], [1, 1]),
          (9, 1, 32, [333, 15], [1, 1]), (16, 1, 16, [77], [1]), (17, 1, 16, [77], [1]), (40, 1, 64, [500], [1]),
          (128, 1, 16, [129, 4], [1, 2]), (6, 2, 48, [200, 31, 64], [5, 8, 3]), (2, 2, 16, [64, 65, 200], [64, 65, 66]),
          (4, 4, 64, [300], [300]), (8, 2, 128, [513, 130], [257, 130]), (3, 1, 16, [1000], [300]),
          (10, 2, 256, [777, 300], [100, 300]), (4, 1, 16, [700, 90, 0, 50, 20], [500, 1, 0, 0, 16]),
          (2, 1, 16, [40] * 37, [1] * 37), (2, 2, 32, [150] * 9, [130, 1, 2, 70, 0, 65, 128, 1, 129]),
          (16, 4, 16, [5000], [1]), (2, 1, 64, [9000], [200])]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("capacity", [0, 2000])  # room for 2,000 rows: key ranges may be divided
def test_attention(lib, shape, int8, causal, capacity):
    h, *rest = shape
    c = pr.Cache(*rest, int8=int8, seed=sum(rest[2]), capacity=capacity).fill()
    for gain in (1.0, 6.0):
        compare(lib, c, queries(c, h, gain), causal)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [1, 4, 17, 200])
def test_strides_of_queries_outputs_and_pages(lib, int8, new):
    """Queries and outputs token by token, as slices of a wider projection, pages as halves of a common pool."""
    c = pr.Cache(2, 16, [300, 210], [new, new], int8=int8, seed=8).fill()
    q = queries(c, 6)
    plain = compare(lib, c, q, True)
    wide = torch.randn(c.N, 10, 64, device="cuda").to(BF)
    wide[:, 2:8] = q.transpose(0, 1)
    out = torch.full((c.N, 7, 64), float("nan"), dtype=BF, device="cuda")
    pool = torch.stack((c.k_pages, c.v_pages), 1)
    c.k_pages, c.v_pages = pool[:, 0], pool[:, 1]
    compare(lib, c, wide[:, 2:8].transpose(0, 1), True, out=out[:, 1:].transpose(0, 1))
    assert torch.equal(out[:, 1:].transpose(0, 1), plain) and torch.all(torch.isnan(out[:, 0]))
    # (max_new has a say in how rows are taken, and so in the last bit)
    free = lib.sdpa_paged_forward(wide[:, 2:8].transpose(0, 1), *c.args, c.row_starts, c.seq_lens, mask="causal", max_new=new,
                                  **c.scales)
    assert bool((free == plain).all())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [1, 3, 100])
@pytest.mark.parametrize("capacity", [0, 2000])
def test_pages_that_are_not_there_are_not_seen(lib, int8, new, capacity):
    """Table entries of -1 and past the pool, at the beginning, inside and for a whole sequence."""
    c = pr.Cache(2, 32, [300, 130, 40, 700], [new, new, min(new, 40), new], int8=int8, seed=9, capacity=capacity).fill()
    gone = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in c.lens]
    for b, i, entry in ((0, 0, -1), (0, 1, -1), (0, 5, c.pages), (1, 4, 1 << 30), (2, 0, -1), (2, 1, -5), (3, 7, -2), (3, 8, -1)):
        c.page_table[b, i] = entry
        gone[b][32 * i:32 * i + 32] = True
    o = compare(lib, c, queries(c, 4), True, gone)
    assert torch.all(o[:, c.starts[2]:c.starts[3]] == 0)
    compare(lib, c, queries(c, 4), False, gone)


@pytest.mark.parametrize("int8", [False, True])
def test_tokens_without_keys_and_rows_of_no_sequence(lib, int8):
    """More new tokens than rows, empty sequences, packed rows in front of the first and behind the last sequence."""
    c = pr.Cache(2, 16, [10, 0, 5, 90], [10, 0, 5, 90], int8=int8, seed=10).fill()
    q = torch.cat((queries(c, 4)[:, :3], queries(c, 4), queries(c, 4)[:, :7]), 1)
    starts = c.row_starts + 3
    out = torch.full_like(q, 5.0)
    for lens, zero in (([10, 0, 5, 90], []), ([4, 0, 5, 30], [(0, 6), (15, 60)]), ([0, 0, 0, 0], [(0, 105)])):
        lib.sdpa_paged_forward(q, *c.args, starts, ints(*lens), out, max_new=90, mask="causal", **c.scales)
        assert torch.all(out[:, :3] == 5) and torch.all(out[:, 3 + c.N:] == 5)
        for first, n in zero:
            assert torch.all(out[:, 3 + first:3 + first + n] == 0)
        assert torch.all(torch.isfinite(out))
    # lengths and starts out of range: clamped, nothing past them is touched
    out.fill_(5.0)
    lib.sdpa_paged_forward(q, *c.args, ints(-4, 3, 3, 8, 9000), ints(-1, 50, 1 << 30, 1 << 30), out, mask="none", **c.scales)
    torch.cuda.synchronize()


@pytest.mark.parametrize("int8", [False, True])
def test_tokens_past_max_new_are_left_out(lib, int8):
    c = pr.Cache(2, 16, [50, 300, 40], [3, 200, 1], int8=int8, seed=11).fill()
    q = queries(c, 4)
    want = compare(lib, c, q, True)
    for most in (2, 60, 150):
        out = lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, torch.full_like(q, 5.0), max_new=most, mask="causal",
                                     **c.scales)
        for b in range(3):
            s, n = c.starts[b], min(c.new[b], most)
            assert (out[:, s:s + n].double() - want[:, s:s + n].double()).abs().max() <= 4 * pr.U * want.abs().max()
            assert torch.all(out[:, s + n:c.starts[b + 1]] == 5)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30])
def test_scales_of_the_scores(lib, int8, scale):
    c = pr.Cache(1, 16, [90, 400], [1, 150], int8=int8, seed=12).fill()
    q = queries(c, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, scale=scale, mask="causal", status=status, **c.scales)
    want, tol = pr.attend(q, c, True, scale)
    ref.check("o", out, want, tol, 0)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [1, 2, 90])
@pytest.mark.parametrize("capacity", [0, 2000])
def test_scores_that_grow_and_shrink_along_the_keys(lib, int8, new, capacity):
    """Scores that rise by thousands towards either end, so that references move at almost every step, and rows far below 0."""
    c = pr.Cache(1, 16, [900, 900, 260], [new, new, new], int8=int8, seed=13, capacity=capacity)
    ramp = torch.linspace(0, 60, 900, device="cuda")
    up = torch.ones(64, device="cuda")
    for b, r in enumerate((ramp, ramp.flip(0), -ramp[:260] - 40)):
        k, v = c.rows[b]
        c.rows[b] = ((k.float() * 0.1 + r[:, None] * up).to(BF), v)
    c.fill()
    q = (queries(c, 2).float() * 0.1 + 1).to(BF)
    compare(lib, c, q, True)
    compare(lib, c, q, False)


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("int8", [False, True])
def test_nan_reaches_what_sees_it_and_nothing_else(lib, new, int8):
    c = pr.Cache(1, 16, [200, 150], [new, new], int8=int8, seed=14)
    c.rows[0][0][0, 37, 5] = float("nan")
    c.fill()
    q = queries(c, 2)
    out = lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, mask="causal", max_new=new, **c.scales)
    assert torch.all(torch.isnan(out[:, :new])) and torch.all(torch.isfinite(out[:, new:]))
    q[0, new, 3] = float("inf")
    out = lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, mask="causal", max_new=new, **c.scales)
    assert torch.all(torch.isnan(out[0, new])) and torch.all(torch.isfinite(out[1, new:]))


def test_small_and_large_magnitudes(lib):
    """Queries, keys and values whose sizes differ by up to 2^60, row by row."""
    for int8 in (False, True):
        c = pr.Cache(1, 16, [300, 280], [1, 130], int8=int8, seed=15)
        for b in range(2):
            k, v = c.rows[b]
            f = torch.exp2(torch.randint(-40, 41, (1, c.lens[b], 1), generator=c.g, device="cuda").float())
            c.rows[b] = ((k.float() * 2.0 ** 30).to(BF), (v.float() * f).to(BF))
        c.fill()
        q = (queries(c, 2).float() * 2.0 ** -30).to(BF)
        compare(lib, c, q, True)


# ------------------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("int8", [False, True])
def test_serving_from_prompt_to_single_tokens(lib, int8):
    """Prompts in chunks, then drafted and single tokens, each appended and attended, equal attention over the whole
    sequences; the rows read back and given to the calls for contiguous caches give the same outputs."""
    h, h_kv, page = 4, 2, 16
    steps = [[100, 40], [70, 0], [1, 33], [3, 1], [1, 1], [1, 1]]
    lens = [sum(s[b] for s in steps) for b in range(2)]
    c = pr.Cache(h_kv, page, lens, [0, 0], int8=int8, seed=16)
    qs = [torch.randn(h, n, 64, generator=c.g, device="cuda").to(BF) for n in lens]
    done, got = [0, 0], [[], []]
    for new in steps:
        part = [slice(done[b], done[b] + new[b]) for b in range(2)]
        k, v = (torch.cat([c.rows[b][i][:, part[b]] for b in range(2)], 1) for i in range(2))
        q = torch.cat([qs[b][:, part[b]] for b in range(2)], 1)
        done = [d + n for d, n in zip(done, new)]
        starts, now = ints(0, new[0], sum(new)), ints(*done)
        lib.paged_cache_append(k, v, *c.args, starts, now, **c.scales)
        o = lib.sdpa_paged_forward(q, *c.args, starts, now, max_new=max(new), mask="causal", **c.scales)
        got[0].append(o[:, :new[0]])
        got[1].append(o[:, new[0]:])
    c.new, c.starts, c.N = lens, [0, lens[0], sum(lens)], sum(lens)
    want, tol = pr.attend(torch.cat(qs, 1), c, True)
    ref.check("o", torch.cat(got[0] + got[1], 1), want, tol, 2)
    k, v = lib.paged_cache_read(*c.args, ints(*lens), rows=256, **c.scales)
    whole = lib.sdpa_scored_forward(torch.nn.functional.pad(qs[0], (0, 0, 0, 256 - lens[0]))[None], k[:1], v[:1], mask="causal")
    ref.check("scored", whole[0, :, :lens[0]], want[:, :lens[0]], tol[:, :lens[0]], 2)
    last = torch.stack([q[:, -1:] for q in qs])
    step = lib.sdpa_decode_forward(last, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1), ints(*lens))
    ends = [lens[0] - 1, sum(lens) - 1]
    for b in range(2):
        ref.check("decode", step[b], want[:, ends[b]:ends[b] + 1], tol[:, ends[b]:ends[b] + 1], 0)


def test_int8_equals_bf16_over_what_is_read_back(lib):
    """Attention over the 8-bit cache and over a bf16 cache of the values read from it: the same function."""
    c = pr.Cache(2, 32, [500, 300, 64], [1, 200, 17], int8=True, seed=17).fill()
    q = queries(c, 4)
    a = compare(lib, c, q, True).double()
    d = pr.Cache(2, 32, c.lens, c.new, seed=17)
    d.rows = [tuple(x.to(BF) for x in c.cached(b)) for b in range(3)]
    d.fill()
    z = compare(lib, d, q, True).double()
    assert (a - z).norm() <= 2 * pr.U * z.norm()


def test_equal_calls_give_equal_bits(lib):
    c = pr.Cache(2, 16, [3000, 700, 40], [1, 300, 4], int8=True, seed=18).fill()
    q = queries(c, 8)
    a = compare(lib, c, q, True)
    for _ in range(10):
        assert torch.equal(a, lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, mask="causal", max_new=300, **c.scales))
