"""Calls that the header allows at its edges: ids that decrease, tables with a type's lowest values, two host threads, a
capture that forks to a stream of its own."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import BF, bias_args, docs, gen, ints, lib, make, run  # noqa: E402,F401


@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
def test_ids_that_decrease_stay_in_range(lib, bias):
    """Which keys are seen is unspecified; nothing is read or written out of range (the status of the checked build), and no
    output is left unwritten."""
    for T in (5, 300, 1500):
        q, k, v, go = make(2, 4, 2, T, T, 121)
        for n, ids in enumerate((torch.randint(-5, 5, (2, T), generator=gen(122), device="cuda", dtype=torch.int32),
                                 torch.arange(T, 0, -1, device="cuda", dtype=torch.int32).expand(2, T).contiguous(),
                                 torch.randint(-2 ** 31, 2 ** 31 - 1, (2, T), generator=gen(123), device="cuda", dtype=torch.int32))):
            form = {"mask": ("causal", "none", "causal_key_padding")[n], "doc_ids": ids, **bias_args(bias, 4, 124, both=n == 1)}
            if "padding" in form["mask"]:
                form["key_lens"] = ints(T // 2, T)
            got = run(lib, q, k, v, go, form)
            for name in ("o", "o2"):
                assert not bool(torch.isnan(got[name].float()).any()), name


def test_ids_of_the_whole_range(lib):
    T = 260
    q, k, v, go = make(1, 2, 2, T, T, 125)
    ids = torch.full((1, T), -2 ** 31, dtype=torch.int32, device="cuda")
    ids[:, 100:] = 2 ** 31 - 1
    form = {"doc_ids": ids}
    want = ref.attention(q, k, v, scale=0.125, dout=go, **form)
    got = run(lib, q, k, v, go, form)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n], want[n + "_tol"], 0)


@pytest.mark.parametrize("lowest", [-float("inf"), torch.finfo(BF).min])
@pytest.mark.parametrize("cap", [None, 20.0])
def test_tables_with_lowest_values(lib, lowest, cap):
    """A bucket of the type's lowest value, or of -infinity, has no weight; a query that sees nothing else outputs 0."""
    T = 330
    q, k, v, go = make(2, 2, 2, T, T, 126)
    starts = (0, 1, 2, 40, 200)
    table = torch.randn(5, 2, generator=gen(127), device="cuda").to(BF)
    for dead in ((3,), (4,), (0,), (1, 2)):
        table_ = table.clone()
        for u in dead:
            table_[u] = lowest
        form = {"mask": "causal", "cap": cap, "table": table_, "bucket_starts": starts}
        got = run(lib, q, k, v, go, form)
        # the definition with those pairs out of sight
        d = torch.arange(T, device="cuda")[None] - torch.arange(T, device="cuda")[:, None]
        b = ref.bucket_of(d, starts, False)
        vis = (d <= 0) & ~sum((b == u) for u in dead).bool()
        s = q.double() @ k.double().transpose(2, 3) * 0.125
        s = cap * torch.tanh(s / cap) if cap else s
        s = torch.where(vis, s + table.double().t()[:, b], -float("inf"))
        lse = torch.logsumexp(s, -1)
        p = torch.where(vis, torch.exp(s - torch.where(lse.isfinite(), lse, 0.0)[..., None]), 0.0)
        want = p @ v.double()
        e = 2 * (2.0 ** -18 * 40 + (6e-4 if cap else 0.0))
        ref.check("o", got["o"], want, (ref.U + e) * (p @ v.double().abs() + want.abs()) + ref.U * want.abs() + 1e-30, 0)
        ref.check("lse", got["lse"], lse, torch.full_like(lse, e), 0)
        for n in ("dq", "dk", "dv", "dtable"):
            assert bool(torch.isfinite(got[n].float()).all()), (n, dead)
        assert torch.all(got["dtable"][list(dead)] == 0)


def test_two_threads(lib):
    q, k, v, go = make(2, 4, 2, 500, 500, 128)
    forms = [{"mask": "causal", "doc_ids": docs(2, 500, 6, 129), **bias_args("buckets", 4, 130)},
             {"mask": "none", "cap": 20.0, **bias_args("slopes", 4, 0)}]
    want = [run(lib, q, k, v, go, f) for f in forms]
    faults = []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    o, lse = lib.sdpa_scored_forward_lse(q, k, v, **forms[n])
                    grads = lib.sdpa_scored_backward(q, k, v, o, go, lse, **forms[n])
                    torch.cuda.current_stream().synchronize()
                    if not (torch.equal(o, want[n]["o2"]) and torch.equal(lse, want[n]["lse"]) and torch.isfinite(grads[0]).all()):
                        faults.append(n)
                    with_lo = (grads[2].double() - want[n]["dv"].double()).norm()
                    if not with_lo <= 2 * ref.U * want[n]["dv"].double().norm():
                        faults.append(n)
        except Exception as e:  # noqa: BLE001
            faults.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(n,)) for n in (0, 1, 0)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults


def test_a_capture_that_forks(lib):
    q, k, v, go = make(2, 4, 2, 300, 300, 131)
    form = {"mask": "causal", **bias_args("buckets", 4, 132)}
    want = run(lib, q, k, v, go, form)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        lo = torch.empty_like(q)
        side.wait_stream(main)
        o, lse = lib.sdpa_scored_forward_lse(q, k, v, out_lo=lo, stream=side, **form)
        dq, dk, dv, dtable = lib.sdpa_scored_backward(q, k, v, o, go, lse, o_lo=lo, stream=side, **form)
        other = lib.sdpa_scored_forward(q, k, v, mask="causal")
        main.wait_stream(side)
    for _ in range(3):
        for t in (o, lse, dk, dv, dtable, other):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for n, t in (("o2", o), ("lse", lse), ("dk", dk), ("dv", dv), ("dtable", dtable)):
            assert torch.equal(t, want[n]), n
        assert torch.isfinite(other).all()
