"""Decoding over a shared prefix (sdpa_decode_shared_forward) against its definition in fp64, and together with the
scored forward that fills its caches."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import bias_args, gen, ints, lib  # noqa: E402,F401

BF = torch.bfloat16


def make(B, h, h_kv, T_q, P, T_k, seed, gain=1.0):
    g = gen(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return ((n(B, h, T_q, 64) * gain).to(BF), n(h_kv, P, 64).to(BF), n(h_kv, P, 64).to(BF), n(B, h_kv, T_k, 64).to(BF),
            n(B, h_kv, T_k, 64).to(BF))


def compare(lib, x, lens, form):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(x[0], float("nan"))
    lib.sdpa_decode_shared_forward(*x, lens, o, status=status, **form)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want, tol = ref.decode(*x, lens, **{**form, "scale": form.get("scale") or 0.125})
    ref.check("o", o, want, tol, 2, x[0].shape[0] * x[0].shape[1] * x[0].shape[2])
    return o


# (B, h, h_kv, T_q, P, T_k): one row, odd sizes, no prefix, no cache, 128 and more stacked rows, many key ranges
SHAPES = [(1, 1, 1, 1, 1, 1), (3, 4, 2, 1, 129, 77), (2, 6, 2, 5, 1000, 33), (5, 3, 3, 8, 64, 200), (2, 2, 2, 3, 0, 50),
          (3, 2, 1, 2, 300, 0), (40, 16, 4, 1, 500, 130), (2, 64, 1, 4, 700, 20), (3, 40, 2, 7, 257, 9),
          (4, 2, 2, 1, 20000, 600)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
@pytest.mark.parametrize("mask", ["none", "causal_key_padding"])
def test_shapes(lib, shape, bias, mask):
    B, h, h_kv, T_q, P, T_k = shape
    x = make(*shape, seed=sum(shape), gain=3.0)
    lens = torch.randint(min(T_q, T_k), T_k + 1, (B,), generator=gen(1), device="cuda", dtype=torch.int32)
    for cap in (None, 10.0):
        form = {"mask": mask, "cap": cap, **bias_args(bias, h, 2, both=B % 2 == 0)}
        compare(lib, x, lens, form)


def test_lengths_past_their_range_and_none(lib):
    x = make(4, 2, 1, 2, 140, 100, 3)
    for mask in ("none", "causal"):
        compare(lib, x, ints(-5, 0, 1, 500), {"mask": mask, **bias_args("slopes", 2, 0)})
        compare(lib, x, None, {"mask": mask, **bias_args("buckets", 2, 4)})


def test_nothing_to_see_outputs_zero(lib):
    x = make(2, 2, 2, 2, 0, 40, 5)
    o = compare(lib, x, ints(0, 40), {})
    assert torch.all(o[0] == 0)


def test_cache_rows_past_the_length_hold_anything(lib):
    x = make(3, 4, 2, 2, 200, 90, 6)
    lens = ints(17, 0, 89)
    a = compare(lib, x, lens, {"cap": 9.0})
    for b, n in enumerate(lens.tolist()):
        x[3][b, :, n:] = float("nan")
        x[4][b, :, n:] = float("nan")
    z = lib.sdpa_decode_shared_forward(*x, lens, cap=9.0)
    assert torch.equal(a, z)


def test_equals_decoding_over_the_whole_sequence(lib):
    """Without a form, the prefix copied in front of every cache gives sdpa_decode_forward's result."""
    B, h, P, T_k = 3, 4, 333, 60
    q, kp, vp, kc, vc = make(B, h, h, 2, P, T_k, 7)
    lens = ints(60, 2, 31)
    whole = [torch.cat((p.expand(B, -1, -1, -1), c), 2).contiguous() for p, c in ((kp, kc), (vp, vc))]
    a = lib.sdpa_decode_shared_forward(q, kp, vp, kc, vc, lens).double()
    b = lib.sdpa_decode_forward(q, *whole, lens + P).double()
    assert (a - b).norm() <= 2 * ref.U * b.norm()


@pytest.mark.parametrize("bias", ["slopes", "buckets"])
def test_prefill_then_decode(lib, bias):
    """The serving path: a prompt of shared tokens and each request's own, by the scored forward; its last rows by a
    decoding step over the prefix and the caches."""
    B, h, h_kv, P, own, T_q = 3, 4, 2, 290, 70, 3
    g = gen(8)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    kp, vp, kc, vc = n(h_kv, P, 64), n(h_kv, P, 64), n(B, h_kv, own, 64), n(B, h_kv, own, 64)
    q = n(B, h, P + own, 64)
    form = {"cap": 15.0, **bias_args(bias, h, 9)}
    k, v = (torch.cat((p.expand(B, -1, -1, -1), c), 2).contiguous() for p, c in ((kp, kc), (vp, vc)))
    full = lib.sdpa_scored_forward(q, k, v, mask="causal", **form)[:, :, P + own - T_q:].double()
    step = lib.sdpa_decode_shared_forward(q[:, :, P + own - T_q:].contiguous(), kp, vp, kc, vc, None, mask="causal", **form)
    assert (full - step.double()).norm() <= 2 * ref.U * full.norm()


def test_training_step_then_serving(lib):
    """Forward, backward and an update of the bias table, then a decoding step with the updated table."""
    B, h, h_kv, T = 2, 4, 2, 200
    g = gen(10)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    q, k, v, go = n(B, h, T, 64), n(B, h_kv, T, 64), n(B, h_kv, T, 64), n(B, h, T, 64)
    form = {"cap": 20.0, **bias_args("buckets", h, 11)}
    lo = torch.empty_like(q)
    o, lse = lib.sdpa_scored_forward_lse(q, k, v, mask="causal", out_lo=lo, **form)
    dq, dk, dv, dtable = lib.sdpa_scored_backward(q, k, v, o, go, lse, mask="causal", o_lo=lo, **form)
    want = ref.attention(q, k, v, scale=0.125, mask="causal", dout=go, **form)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv), ("dtable", dtable)):
        ref.check(name, got, want[name], want[name + "_tol"], 0 if name == "dtable" else 2)
    form["table"] = (form["table"].float() - 0.1 * dtable.float()).to(BF)
    x = make(B, h, h_kv, 1, 150, 40, 12)
    compare(lib, x, ints(40, 13), form)


def test_streams_and_graphs(lib):
    x = make(4, 8, 2, 2, 900, 100, 13)
    lens = ints(100, 2, 50, 77)
    forms = [{"mask": "causal", **bias_args("buckets", 8, s)} for s in (14, 15)]
    want = [lib.sdpa_decode_shared_forward(*x, lens, **f) for f in forms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in forms]
    for _ in range(5):
        got = []
        for s, f in zip(streams, forms):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(lib.sdpa_decode_shared_forward(*x, lens, **f))
        torch.cuda.synchronize()
        assert all(torch.equal(a, z) for a, z in zip(want, got))
    graphs = []
    for f in forms:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = lib.sdpa_decode_shared_forward(*x, lens, **f)
        graphs.append((graph, out))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, out) for a, (_, out) in zip(want, graphs))


@pytest.mark.parametrize("B,T_k", [(128, 40), (129, 40), (300, 700), (5, 3000)])
def test_batches_of_single_rows(lib, B, T_k):
    """Batches that are ordered by length and ones too large for that, equal lengths and empty caches among them."""
    x = make(B, 2, 2, 1, 200, T_k, 41)
    lens = torch.randint(0, T_k + 1, (B,), generator=gen(42), device="cuda", dtype=torch.int32)
    lens[1::3] = lens[1]
    lens[::4] = 0
    compare(lib, x, lens, {"mask": "key_padding", **bias_args("slopes", 2, 43)})


@pytest.mark.parametrize("h_kv,T_q", [(8, 1), (2, 1), (4, 3)])
@pytest.mark.parametrize("biased", [False, True])
def test_inputs_written_just_before(lib, h_kv, T_q, biased):
    """The caches, the query and the lengths are written right before each call and destroyed right after it, eagerly and
    captured: launches may overlap the ends of the ones before them."""
    B, h, P, T_k = 48, 8, 3000, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    source = [n(B, h, T_q, 64), n(h_kv, P, 64), n(h_kv, P, 64), n(B, h_kv, T_k, 64), n(B, h_kv, T_k, 64)]
    lens = torch.randint(T_q, T_k + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    form = {"table": n(16, h), "bucket_starts": lib.relative_bucket_starts(16, 128)} if biased else {}
    want = lib.sdpa_decode_shared_forward(*source, lens, **form)
    x, m = [torch.empty_like(t) for t in source], torch.empty_like(lens)

    def step():
        out = []
        for _ in range(3):
            for t, f in zip(x, source):
                t.copy_(f)
            torch.add(lens, 0, out=m)
            out.append(lib.sdpa_decode_shared_forward(*x, m, **form))
            for t in x:
                t.fill_(float("nan"))
            m.zero_()
        return out

    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in eager + captured:
        assert torch.equal(o, want)


def test_refusals(lib):
    q, kp, vp, kc, vc = make(2, 4, 2, 9, 20, 10, 16)
    with pytest.raises(lib.MhaError):  # more rows than a decoding step has
        lib.sdpa_decode_shared_forward(q, kp, vp, kc, vc)
    q = q[:, :, :1].contiguous()
    with pytest.raises(ValueError):
        lib.sdpa_decode_shared_forward(q, kp[:1], vp, kc, vc)
    with pytest.raises(ValueError):
        lib.sdpa_decode_shared_forward(q, kp, vp, kc, vc, ints(1))
    with pytest.raises(lib.MhaError):
        lib.sdpa_decode_shared_forward(q, kp, vp, kc, vc, mask="key_padding")
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(lib.MhaError):
        lib.sdpa_decode_shared_forward(q, kp, vp, kc, vc, workspace=small)
