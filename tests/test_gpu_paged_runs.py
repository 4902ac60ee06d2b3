"""Chunks over so many cached rows that a row tile's key tiles are summed in several runs: fp32 sums in the tensor cores drop
what lies below an addend's place in them, which one long run turns into a bias."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402
import scored_reference as ref  # noqa: E402
from test_gpu_paged import BF, ints, lib  # noqa: E402,F401
from test_gpu_scored_windows import SCALE, keys, rows  # noqa: E402

PAGE = 1 << 16


@pytest.mark.parametrize("int8,table", [(False, 1 << 22), (True, 1 << 22), (True, 1 << 25)])  # straight, laid out first, straight
@pytest.mark.parametrize("length", [1 << 16, (1 << 20) + 777, 1 << 22, 1 << 24])
def test_values_of_one_sign_over_many_rows(lib, int8, table, length):
    """One page of 65,536 rows, over and over: softmax over k copies of a set of keys is that over the set (the first 777 of
    them once more are part of the sum).  Values between 0.5 and 1: nothing cancels."""
    g = torch.Generator(device="cuda").manual_seed(61)
    k, v = torch.randn(PAGE, 64, generator=g, device="cuda").to(BF), (torch.rand(PAGE, 64, generator=g, device="cuda") / 2 + 0.5).to(BF)
    c = pr.Cache(1, PAGE, [PAGE], [0], int8=int8, seed=61, spare=0)
    c.rows = [(k[None], v[None])]
    c.fill()
    k, v = (x[0] for x in c.cached(0))
    N, h = 1024, 16
    q = torch.randn(h, N, 64, generator=g, device="cuda").to(BF)
    pages = torch.full((1, max(table, length) // PAGE), -1, dtype=torch.int32, device="cuda")
    pages[:, :-(-length // PAGE)] = 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.sdpa_paged_forward(q, c.k_pages, c.v_pages, pages, ints(0, N), ints(length), status=status, **c.scales)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    some = q[:, ::61].double()
    s = some @ k.t() * 0.125
    w = torch.exp(s - s.amax(-1, keepdim=True)) * (length // PAGE + (torch.arange(PAGE, device="cuda") < length % PAGE))
    w = w / w.sum(-1, keepdim=True)
    want = w @ v
    e = 2 * ref.score_error(None, 0.125 * (some.abs() @ k.abs().t())).amax(-1, keepdim=True)
    ref.check("o", out[:, ::61], want, (ref.U + e) * 2 * want + ref.U * want, 0)


# tiles of 128 keys, in runs of 1,024 from the last one down: references that differ between runs, and a run without weight
TILES = {"apart": "A" * 1100 + "B" * 1100, "one each": "B" * 1024 + "A" * 1025, "nothing first": "C" * 1400 + "AB" * 400,
         "nothing last": "D" + "C" * 2100, "one more": "B" * 1025}


@pytest.mark.parametrize("name", list(TILES))
@pytest.mark.parametrize("int8", [False, True])
def test_runs_of_one_row_tile(lib, name, int8):
    tiles = TILES[name]
    n, N, h = 128 * len(tiles), 1280, 16
    c = pr.Cache(1, 128, [n], [N], int8=int8, seed=62, capacity=n if not int8 else 1 << 25)
    g = torch.Generator(device="cuda").manual_seed(62)
    c.rows = [keys(tiles, g, (1,))]
    c.fill()
    q = rows(g, h, N)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, mask="causal", scale=SCALE, status=status, **c.scales)

    out = call()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, call())
    k, v = (x[0] for x in c.cached(0))
    at = torch.arange(0, N, 29, device="cuda")
    some = q[:, at].double()
    vis = torch.arange(n, device="cuda")[None] <= (n - N + at)[:, None]
    w, _, _, _ = ref.weights(some @ k.t() * SCALE, None, 0.0, vis[None])
    e = 2 * ref.score_error(None, SCALE * (some.abs() @ k.abs().t())).amax(-1, keepdim=True)
    want = w @ v
    ref.check("o", out[:, at], want, (ref.U + e) * (w @ v.abs() + want.abs()) + ref.U * want.abs() + 2.0 ** -51 * v.abs().max(), 0)


@pytest.mark.parametrize("int8", [False, True])
def test_a_key_far_ahead_in_another_run(lib, int8):
    """A single key with all of the weight, in the first, a middle and the last run, and none with more than the others."""
    n, N, h = 128 * 2100, 1280, 16
    c = pr.Cache(1, 128, [n], [N], int8=int8, seed=63, capacity=n if not int8 else 1 << 25)
    g = torch.Generator(device="cuda").manual_seed(63)
    q = rows(g, h, N)
    for at in (3, 128 * 1090 + 5, n - N):
        k, v = torch.zeros(1, n, 64, device="cuda"), torch.randn(1, n, 64, generator=g, device="cuda")
        k[0, at, 0] = 40.0
        c.rows = [(k.to(BF), v.to(BF))]
        c.fill()
        out = lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, mask="causal", scale=SCALE, **c.scales)
        want = c.cached(0)[1][0, at]
        # the others have 2^-40 each, 2^-21.9 together
        assert (out.double() - want).abs().max() <= ref.U * want.abs().max() + 2.0 ** -20


# Few query rows: a warp's own sum is as long only where the batch's rows are many times those that fit a GPU: pages of 4,096
# rows that sequences share.
def shared(c, q, table, lens, scale):
    """(o, bound) of single tokens q (h, B, 64), from what the pages hold and how often each row counts."""
    g = q.shape[0] // c.h_kv
    k, v = (torch.stack([c.cached(b)[i] for b in range(c.B)]).transpose(0, 1).reshape(c.h_kv, -1, 64).repeat_interleave(g, 0)
            for i in range(2))
    which = torch.empty(c.pages, dtype=torch.long, device="cuda")
    which[c.page_table[:, 0].long()] = torch.arange(c.B, device="cuda")
    times = torch.zeros(q.shape[1], c.B, c.page, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        whole, rest = divmod(n, c.page)
        times[b] = torch.bincount(which[table[b, :whole].long()], minlength=c.B).double()[:, None]
        if rest:
            times[b, which[table[b, whole].long()], :rest] += 1
    s = q.double() @ k.transpose(1, 2) * scale
    times = times.reshape(len(lens), -1)
    w = torch.where(times > 0, torch.exp(s - torch.where(times > 0, s, -math.inf).amax(-1, keepdim=True)), 0.0) * times
    w = w / w.sum(-1, keepdim=True)
    e = 2 * ref.score_error(None, abs(scale) * (q.double().abs() @ k.abs().transpose(1, 2))).amax(-1, keepdim=True)
    o = w @ v
    return o, (ref.U + e) * (w @ v.abs() + o.abs()) + ref.U * o.abs() + 2.0 ** -51 * v.abs().max()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("g", [1, 9, 20])
def test_single_tokens_over_many_rows_of_one_sign(lib, int8, g):
    if g == 20 and not int8:
        g = 16
    B, h_kv, length, page = 64, 16, (1 << 22) + 1000, 4096
    c = pr.Cache(h_kv, page, [page], [0], int8=int8, seed=64, spare=0)
    c.rows = [(c.rows[0][0], (torch.rand(h_kv, page, 64, generator=c.g, device="cuda") / 2 + 0.5).to(BF))]
    c.fill()
    q = torch.randn(g * h_kv, B, 64, generator=c.g, device="cuda").to(BF)
    table = torch.zeros(B, length // page + 1, dtype=torch.int32, device="cuda")
    out = lib.sdpa_paged_forward(q, c.k_pages, c.v_pages, table, torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                                 ints(*[length] * B), max_new=1, **c.scales)
    ref.check("o", out, *shared(c, q, table, [length] * B, 0.125), 0)
    mean = ((out.double() - shared(c, q, table, [length] * B, 0.125)[0]).mean() / 0.75).item()
    # outputs near 0.75 are rounded to multiples of 2^-8: half a step at most were they all alike
    assert abs(mean) <= 2.0 ** -9


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("orders", [["ABC", "BAC", "CAB", "CBA"], ["AAB", "BBA", "BCB", "ACA"]])
def test_single_tokens_whose_references_differ_between_runs(lib, int8, orders):
    h_kv, page, h = 16, 4096, 32
    c = pr.Cache(h_kv, page, [page] * 3, [0] * 3, int8=int8, seed=65, spare=0)
    g = torch.Generator(device="cuda").manual_seed(65)
    c.rows = [keys(t * (page // 128), g, (h_kv,)) for t in "ABC"]
    c.fill()
    lens = [3 * 400 * page - 7 * b for b in range(4)]
    table = torch.stack([torch.cat([c.page_table["ABC".index(t), 0].repeat(400) for t in o]) for o in orders]).contiguous()
    q, starts = rows(g, h, 4), ints(0, 1, 2, 3, 4)

    def call():
        return lib.sdpa_paged_forward(q, c.k_pages, c.v_pages, table, starts, ints(*lens), max_new=1, scale=SCALE, **c.scales)

    out = call()
    assert torch.equal(out, call())
    ref.check("o", out, *shared(c, q, table, lens, SCALE), 0)
