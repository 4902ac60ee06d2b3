"""Scored attention (sdpa_scored_forward / _backward) against its definition in fp64, elementwise within bounds derived
from the roundings (scored_reference.py)."""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    import transformer_scaled_dot_softmax_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(B, h, h_kv, T_q, T_k, seed, gain=1.0):
    g = gen(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return ((n(B, h, T_q, 64) * gain).to(BF), n(B, h_kv, T_k, 64).to(BF), n(B, h_kv, T_k, 64).to(BF),
            n(B, h, T_q, 64).to(BF))


def bias_args(kind, h, seed, both=False, starts=None):
    if kind == "slopes":
        return {"slopes": torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")}
    if kind == "buckets":
        import transformer_scaled_dot_softmax_gb300 as m
        starts = starts or m.relative_bucket_starts(16, 128)
        return {"bucket_starts": starts,
                "table": torch.randn(len(starts) * (2 if both else 1), h, generator=gen(seed), device="cuda").to(BF)}
    return {}


def docs(B, T, n, seed):
    cuts = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    if T > 1 and n > 1:
        cuts.scatter_(1, torch.randint(1, T, (B, n - 1), generator=gen(seed), device="cuda"), 1)
    return torch.cumsum(cuts, 1, dtype=torch.int32)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(lib, q, k, v, go, form, o_lo=True):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, float("nan"))
    lib.sdpa_scored_forward(q, k, v, o, status=status, **form)
    lo = torch.full_like(q, float("nan")) if o_lo else None
    o2, lse = lib.sdpa_scored_forward_lse(q, k, v, out_lo=lo, status=status, **form)
    grads = {"dq": torch.full_like(q, float("nan")), "dk": torch.full_like(k, float("nan")),
             "dv": torch.full_like(v, float("nan"))}
    dq, dk, dv, dtable = lib.sdpa_scored_backward(q, k, v, o2, go, lse, o_lo=lo, status=status, **grads, **form)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return {"o": o, "o2": o2, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}


def compare(lib, q, k, v, go, form):
    got = run(lib, q, k, v, go, form)
    scale = form.get("scale") or 0.125
    want = ref.attention(q, k, v, dout=go, **{**form, "scale": scale})
    rows = q.shape[0] * q.shape[1] * q.shape[2]
    fine = ref.attention(q, k, v, two_parts=True, **{**form, "scale": scale})
    ref.check("o2", got["o2"], fine["o"], fine["o_tol"], 1, rows)
    # o: weights and output rounded; gradients: P or dS, and the output
    for n, m, roundings in (("o", "o", 2), ("lse", "lse", 1), ("dq", "dq", 2), ("dk", "dk", 2), ("dv", "dv", 2),
                            ("dtable", "dtable", 0)):
        if got[n] is None:
            assert m not in want
            continue
        ref.check(n, got[n], want[m], want[m + "_tol"], roundings, rows)
    return got, want


SHAPES = [(1, 1, 1, 1, 1), (1, 2, 1, 5, 5), (2, 3, 3, 64, 64), (1, 4, 2, 129, 129), (2, 2, 2, 257, 257),
          (1, 6, 2, 700, 700)]
CROSS = [(1, 1, 1, 1, 300), (1, 2, 1, 130, 1), (2, 3, 1, 100, 513), (1, 2, 2, 600, 90)]


@pytest.mark.parametrize("cap", [None, 30.0])
@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
@pytest.mark.parametrize("mask", ["none", "causal", "key_padding", "causal_key_padding"])
def test_forms_and_shapes(lib, cap, bias, mask):
    for n, (B, h, h_kv, T_q, T_k) in enumerate(SHAPES + CROSS):
        q, k, v, go = make(B, h, h_kv, T_q, T_k, 10 + n, gain=4.0 if cap else 1.0)
        form = {"mask": mask, "cap": cap, **bias_args(bias, h, 40 + n, both=n % 2 == 0)}
        if "key_padding" in mask:
            form["key_lens"] = torch.randint(0, T_k + 1, (B,), generator=gen(n), device="cuda", dtype=torch.int32)
        compare(lib, q, k, v, go, form)


@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
@pytest.mark.parametrize("T", [7, 128, 300, 1025])
def test_documents(lib, bias, T):
    q, k, v, go = make(2, 4, 2, T, T, T)
    for mask in ("none", "causal", "causal_key_padding"):
        form = {"mask": mask, "doc_ids": docs(2, T, 9, T + 1), **bias_args(bias, 4, 5, both=mask == "none")}
        if "padding" in mask:
            form["key_lens"] = ints(T // 3, T)
        compare(lib, q, k, v, go, form)


def test_documents_of_one_token_and_of_all(lib):
    T = 260
    q, k, v, go = make(2, 2, 2, T, T, 77)
    ids = torch.stack((torch.arange(T, device="cuda", dtype=torch.int32), torch.zeros(T, device="cuda", dtype=torch.int32)))
    got, _ = compare(lib, q, k, v, go, {"doc_ids": ids})
    # a token alone in its document sees itself with weight 1
    assert torch.equal(got["o"][0], v[0])


@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
def test_prefixes(lib, bias):
    T = 400
    q, k, v, go = make(5, 2, 1, T, T, 3)
    form = {"mask": "causal", "prefix_lens": ints(-3, 0, 1, 201, 5000), **bias_args(bias, 2, 6, both=True)}
    compare(lib, q, k, v, go, form)
    form.update(mask="causal_key_padding", key_lens=ints(400, 0, 130, 150, 399))
    compare(lib, q, k, v, go, form)
    form.update(doc_ids=docs(5, T, 4, 8))
    compare(lib, q, k, v, go, form)


def test_prefix_of_a_cross_shape(lib):
    q, k, v, go = make(2, 2, 2, 150, 700, 4)
    compare(lib, q, k, v, go, {"mask": "causal", "prefix_lens": ints(300, 650)})


@pytest.mark.parametrize("cap,gain", [(0.5, 1.0), (5.0, 8.0), (50.0, 30.0)])
def test_scores_past_the_cap(lib, cap, gain):
    q, k, v, go = make(1, 2, 2, 200, 200, 9, gain=gain)
    compare(lib, q, k, v, go, {"cap": cap, "mask": "causal"})


@pytest.mark.parametrize("starts", [(0,), (0, 1), (0, 3, 200), tuple(range(64)), (0, 1, 5000)])
@pytest.mark.parametrize("both", [False, True])
def test_bucket_borders(lib, starts, both):
    q, k, v, go = make(2, 3, 1, 390, 390, 21)
    compare(lib, q, k, v, go, {"mask": "none" if both else "causal", **bias_args("buckets", 3, 22, both, starts)})


def test_steep_slopes_and_unequal_ones(lib):
    q, k, v, go = make(1, 3, 3, 513, 513, 31)
    for mask in ("none", "causal"):
        compare(lib, q, k, v, go, {"mask": mask, "slopes": torch.tensor([8.0, 0.0, -0.01], device="cuda")})


def test_slopes_where_only_far_keys_are_seen(lib):
    # rows far past the key length: every bias is large, only differences count
    q, k, v, _ = make(1, 1, 1, 3000, 3000, 32)
    form = {"mask": "key_padding", "key_lens": ints(70), "slopes": torch.tensor([0.5], device="cuda")}
    want = ref.attention(q, k, v, scale=0.125, **form)
    got = lib.sdpa_scored_forward(q, k, v, **form)
    ref.check("o", got, want["o"], want["o_tol"], 2)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_other_scales(lib, scale):
    q, k, v, go = make(1, 2, 2, 140, 140, 33)
    for cap in (None, 4.0):
        form = {"mask": "causal", "cap": cap, "scale": scale}
        got = run(lib, q, k, v, go, form)
        want = ref.attention(q, k, v, dout=go, **form)
        for n, m in (("o", "o"), ("o2", "o"), ("dq", "dq"), ("dk", "dk"), ("dv", "dv")):
            ref.check(n, got[n], want[m], want[m + "_tol"], 2)


def test_rows_that_see_nothing(lib):
    q, k, v, go = make(3, 2, 2, 150, 150, 34)
    form = {"mask": "key_padding", "key_lens": ints(0, 77, 150), "cap": 20.0}
    got, _ = compare(lib, q, k, v, go, form)
    for n in ("o", "o2", "dq", "dk", "dv"):
        assert torch.all(got[n][0] == 0), n
    assert torch.all(got["lse"][0] == float("-inf"))
    assert torch.all(got["dk"][1, :, 77:] == 0) and torch.all(got["dv"][1, :, 77:] == 0)


def test_no_keys_and_no_queries(lib):
    q, _, _, go = make(2, 2, 1, 3, 3, 35)
    empty = torch.empty(2, 1, 0, 64, dtype=BF, device="cuda")
    b = bias_args("buckets", 2, 36)
    o, lse = lib.sdpa_scored_forward_lse(q, empty, empty, **b)
    dq, dk, dv, dtable = lib.sdpa_scored_backward(q, empty, empty, o, go, lse, **b)
    assert torch.all(o == 0) and torch.all(lse == float("-inf")) and torch.all(dq == 0) and torch.all(dtable == 0)
    _, k, v, _ = make(2, 2, 1, 3, 5, 37)
    e = torch.empty(2, 2, 0, 64, dtype=BF, device="cuda")
    o, lse = lib.sdpa_scored_forward_lse(e, k, v, **b)
    dq, dk, dv, dtable = lib.sdpa_scored_backward(e, k, v, o, e, lse, **b)
    assert o.shape == e.shape and torch.all(dk == 0) and torch.all(dv == 0) and torch.all(dtable == 0)
    none = [torch.empty(0, n, 3, 64, dtype=BF, device="cuda") for n in (2, 1, 1)]
    o, lse = lib.sdpa_scored_forward_lse(*none, **b)
    assert torch.all(lib.sdpa_scored_backward(*none, o, o, lse, **b)[3] == 0)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("bias,cap", [("none", None), ("slopes", 30.0), ("buckets", None)])
def test_padding_holds_anything(lib, fill, bias, cap):
    q, k, v, go = make(2, 2, 1, 300, 300, 38)
    lens = ints(130, 257)
    form = {"mask": "causal_key_padding", "key_lens": lens, "cap": cap, **bias_args(bias, 2, 39)}
    a = run(lib, q, k, v, go, form)
    for b, n in enumerate(lens.tolist()):
        k[b, :, n:] = fill
        v[b, :, n:] = fill
    z = run(lib, q, k, v, go, form)
    for n in ("o", "o2", "lse", "dk", "dv"):
        assert torch.equal(a[n], z[n]), n
    if bias == "buckets":
        assert torch.equal(a["dtable"], z["dtable"])
    assert torch.isfinite(z["dq"].float()).all()


def test_equal_calls_give_equal_sums(lib):
    q, k, v, go = make(2, 4, 2, 700, 700, 41)
    form = {"mask": "causal", "cap": 20.0, **bias_args("buckets", 4, 42)}
    a, z = run(lib, q, k, v, go, form), run(lib, q, k, v, go, form)
    for n in ("o", "o2", "lse", "dk", "dv", "dtable"):
        assert torch.equal(a[n], z[n]), n


def test_without_a_form_it_is_sdpa(lib):
    q, k, v, _ = make(2, 3, 3, 333, 333, 43)
    a = lib.sdpa_scored_forward(q, k, v, mask="causal").double()
    b = lib.sdpa_forward(q, k, v, mask="causal").double()
    assert (a - b).norm() <= 2 * ref.U * (2 / 3) ** 0.5 * b.norm()


def test_backward_without_the_remainder(lib):
    q, k, v, go = make(2, 4, 2, 260, 260, 61, gain=3.0)
    form = {"mask": "causal", "cap": 20.0, **bias_args("buckets", 4, 62)}
    got = run(lib, q, k, v, go, form, o_lo=False)
    want = ref.attention(q, k, v, scale=0.125, dout=go, o_lo=False, **form)
    for n in ("dq", "dk", "dv", "dtable"):
        off = (got[n].double() - want[n]).abs()
        assert (off <= want[n + "_tol"]).all(), n


@pytest.mark.parametrize("what", ["q", "k", "v", "table"])
def test_gradients_against_differences(lib, what):
    """(L(x + e d) - L(x - e d)) / 2e of L = sum o dout, exact in fp64, against <gradient, d>."""
    q, k, v, go = make(1, 4, 2, 90, 90, 44, gain=3.0)
    b = bias_args("buckets", 4, 45)
    form = {"mask": "causal", "cap": 6.0, **b}
    got = run(lib, q, k, v, go, form)
    x = {"q": q, "k": k, "v": v, "table": b["table"]}
    g = gen(46)
    d = torch.randn(x[what].shape, generator=g, device="cuda", dtype=torch.float64)

    def loss(e):
        y = {n: t.double() + (e * d if n == what else 0) for n, t in x.items()}
        f = {**form, "table": y["table"], "scale": 0.125}
        return (ref.attention(y["q"], y["k"], y["v"], **f)["o"] * go.double()).sum().item()

    e = 1e-5
    slope = (loss(e) - loss(-e)) / (2 * e)
    grad = got["d" + what].double()
    # the gradient's own relative 2-norm error, at most u sqrt(3/3), times the direction's length
    assert abs((grad * d).sum().item() - slope) <= ref.U * grad.norm().item() * d.norm().item()


def test_largest_length_on_sampled_rows(lib):
    """T = 16,384 causal with slopes and a cap: the last rows against fp64."""
    T = 16384
    q, k, v, _ = make(1, 2, 1, T, T, 47, gain=3.0)
    s = torch.tensor([0.25, 0.001], device="cuda")
    o = lib.sdpa_scored_forward(q, k, v, mask="causal", cap=30.0, slopes=s)
    n = 64
    i, j = torch.arange(T - n, T, device="cuda")[:, None], torch.arange(T, device="cuda")[None]
    ke, ve = (x.double().repeat_interleave(2, 1) for x in (k, v))
    qq = q[:, :, T - n:].double()
    bias = ref.bias_of(j - i, 2, s, None, None)
    p, _, _, _ = ref.weights(qq @ ke.transpose(2, 3) * 0.125, 30.0, bias, j <= i)
    want = p @ ve
    e = 2 * ref.score_error(30.0, (qq.abs() @ ke.abs().transpose(2, 3) * 0.125 + bias.abs()).amax(-1, keepdim=True))
    ref.check("o", o[:, :, T - n:], want, (ref.U + e) * (p @ ve.abs() + want.abs()) + ref.U * want.abs() + 1e-30, 2)


def test_streams_graphs_and_two_calls_at_once(lib):
    q, k, v, go = make(2, 4, 2, 500, 500, 48)
    forms = [{"mask": "causal", "doc_ids": docs(2, 500, 6, 49), **bias_args("buckets", 4, 50)},
             {"mask": "none", "doc_ids": docs(2, 500, 3, 51), **bias_args("buckets", 4, 52, both=True)}]

    def step(form):
        o, lse = lib.sdpa_scored_forward_lse(q, k, v, **form)
        return (o, lse) + lib.sdpa_scored_backward(q, k, v, o, go, lse, **form)

    want = [step(f) for f in forms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in forms]
    for _ in range(3):  # in two streams at once, a workspace each
        got = []
        for s, f in zip(streams, forms):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(f))
        torch.cuda.synchronize()
    graphs = []
    for f in forms:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(f)
        graphs.append((graph, out))
    for _ in range(2):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for results in (got, [o for _, o in graphs]):
        for a, z in zip(want, results):
            for n, x, y in zip(("o", "lse", "dq", "dk", "dv", "dtable"), a, z):
                if n == "dq":  # added up in no fixed order
                    assert (x.double() - y.double()).norm() <= ref.U * x.double().norm()
                else:
                    assert torch.equal(x, y), n


def test_shared_heads_equal_repeated_heads(lib):
    q, k, v, go = make(2, 6, 2, 300, 300, 53)
    form = {"mask": "causal", **bias_args("slopes", 6, 0)}
    a = run(lib, q, k, v, go, form)
    b = run(lib, q, k.repeat_interleave(3, 1).contiguous(), v.repeat_interleave(3, 1).contiguous(), go, form)
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
    for n in ("dk", "dv"):
        x, y = a[n].double(), b[n].double().reshape(2, 2, 3, 300, 64).sum(2)
        assert (x - y).norm() <= 2 * ref.U * y.norm()


def test_many_items_per_processor(lib):
    """More work items than the on-chip item table holds, of two lengths."""
    q, k, v, _ = make(150, 136, 8, 4, 4, 54)
    lens = torch.randint(0, 5, (150,), generator=gen(55), device="cuda", dtype=torch.int32)
    form = {"mask": "causal_key_padding", "key_lens": lens, "cap": 10.0}
    o = lib.sdpa_scored_forward(q, k, v, **form)
    want = ref.attention(q, k, v, scale=0.125, **form)
    ref.check("o", o, want["o"], want["o_tol"], 2)


def test_inputs_written_just_before(lib):
    """Each call's inputs come from work queued right before it (a kernel, a copy, a fill, another stream), eagerly and
    captured, and each output is overwritten right after it: launches may overlap the ends of the ones before them."""
    q, k, v, go = make(2, 4, 2, 700, 700, 95)
    ids = docs(2, 700, 5, 96)
    forms = [{"mask": "causal"}, {"mask": "causal", "doc_ids": ids.clone(), **bias_args("buckets", 4, 97)}]
    x, y, z, g = (torch.empty_like(t) for t in (q, k, v, go))
    o, lo = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()

    def step(form):
        out = []
        for turn in range(3):
            if turn:  # what the turn before used is destroyed
                for t in (x, y, z, g, o, lo):
                    t.fill_(float("nan")) if turn == 1 else t.zero_()
            if "doc_ids" in form:
                form["doc_ids"].zero_()
                form["doc_ids"].copy_(ids)
            torch.mul(q, 1.0, out=x)
            y.copy_(k)
            g.copy_(go)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                z.copy_(v)
            torch.cuda.current_stream().wait_stream(side)
            _, lse = lib.sdpa_scored_forward_lse(x, y, z, o, out_lo=lo, **form)
            dq, dk, dv, dtable = lib.sdpa_scored_backward(x, y, z, o, g, lse, o_lo=lo, **form)
            out.append([o.clone(), lse, dk, dv, dq] + ([] if dtable is None else [dtable]))
        return out

    for form in forms:
        lo_want = torch.empty_like(q)
        o_want, lse_want = lib.sdpa_scored_forward_lse(q, k, v, out_lo=lo_want, **form)
        dq, dk, dv, dtable = lib.sdpa_scored_backward(q, k, v, o_want, go, lse_want, o_lo=lo_want, **form)
        torch.cuda.synchronize()
        want = [o_want, lse_want, dk, dv]
        graph = torch.cuda.CUDAGraph()
        eager = step(form)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            captured = step(form)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for got in eager + captured:
            for a, b in zip(want, got):
                assert torch.equal(a, b)
            assert (dq.double() - got[4].double()).norm() <= ref.U * dq.double().norm()  # added up in no fixed order
            assert dtable is None or torch.equal(dtable, got[5])


@pytest.mark.parametrize("h_kv,bias,cap,mask", [(8, "buckets", None, "causal_key_padding"), (8, "buckets", 20.0, "key_padding"),
                                                (8, "slopes", None, "documents"), (2, "buckets", None, "causal_key_padding"),
                                                (4, "none", 20.0, "key_padding")])
def test_gradients_of_many_items(lib, h_kv, bias, cap, mask):
    # several key blocks for each processor one after the other, blocks that no query sees among them
    B, T = (40, 260) if h_kv == 8 else (120, 390)
    q, k, v, go = make(B, 8, h_kv, T, T, 91)
    form = {"mask": "causal" if mask == "documents" else mask, "cap": cap, **bias_args(bias, 8, 92, both=mask == "key_padding")}
    if mask == "documents":
        form["doc_ids"] = docs(B, T, 6, 93)
    else:
        lens = torch.randint(0, T + 1, (B,), generator=gen(94), device="cuda", dtype=torch.int32)
        lens[::5] = 0
        lens[1::7] = 100
        form["key_lens"] = lens
    compare(lib, q, k, v, go, form)


def test_refusals(lib):
    q, k, v, go = make(1, 4, 2, 8, 8, 56)
    bad = [({"slopes": torch.zeros(3, device="cuda")}, ValueError), ({"slopes": torch.zeros(4, device="cuda").half()}, ValueError),
           ({"table": torch.zeros(4, 4, device="cuda", dtype=BF)}, ValueError),
           ({"table": torch.zeros(3, 4, device="cuda", dtype=BF), "bucket_starts": (0, 2)}, ValueError),
           ({"doc_ids": torch.zeros(1, 7, device="cuda", dtype=torch.int32)}, ValueError),
           ({"prefix_lens": ints(3)}, lib.MhaError), ({"cap": -1.0}, lib.MhaError),
           ({"table": torch.zeros(2, 4, device="cuda", dtype=BF), "bucket_starts": (0, 0)}, lib.MhaError),
           ({"key_lens": ints(1, 2), "mask": "key_padding"}, ValueError), ({"mask": "key_padding"}, lib.MhaError)]
    for form, error in bad:
        with pytest.raises(error):
            lib.sdpa_scored_forward(q, k, v, **form)
    with pytest.raises(ValueError):
        lib.sdpa_scored_forward(q, k.transpose(1, 2), v)
    with pytest.raises(ValueError):
        lib.sdpa_scored_forward(q.float(), k, v)
    with pytest.raises(lib.MhaError):  # 4 heads over 3
        lib.sdpa_scored_forward(q, k[:, :1].repeat(1, 3, 1, 1), v[:, :1].repeat(1, 3, 1, 1))


def test_small_draws(lib):
    """Every pair of (cap, bias, extra mask) over random odd shapes."""
    import random
    rng = random.Random(7)
    for n, (cap, bias, extra) in enumerate(itertools.product((None, 20.0), ("none", "slopes", "buckets"),
                                                            ("none", "prefix", "docs", "both"))):
        B, h_kv, g, T = rng.randint(1, 4), rng.randint(1, 3), rng.choice((1, 2, 5)), rng.randint(2, 450)
        q, k, v, go = make(B, h_kv * g, h_kv, T, T, 100 + n, gain=3.0)
        form = {"mask": "causal", "cap": cap, **bias_args(bias, h_kv * g, 200 + n, both=rng.random() < 0.5)}
        if extra in ("prefix", "both"):
            form["prefix_lens"] = torch.randint(0, T, (B,), generator=gen(n), device="cuda", dtype=torch.int32)
        if extra in ("docs", "both"):
            form["doc_ids"] = docs(B, T, rng.randint(1, 6), n)
        compare(lib, q, k, v, go, form)
