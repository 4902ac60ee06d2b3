"""Calls that are a host thread's first use of CUDA: everything allocated by another thread, no context in this one yet."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    import transformer_scaled_dot_softmax_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def calls(m):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    q, k, v, w = n(1, 2, 300, 64), n(1, 2, 300, 64), n(1, 2, 300, 64), [n(128, 128) for _ in range(4)]
    x, lse = n(1, 300, 128), torch.empty(1, 2, 300, device="cuda")
    c = pr.Cache(2, 16, [300, 90], [200, 1], capacity=2000).fill()
    pq, ws = n(4, c.N, 64), torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return {"forward": lambda o: m.sdpa_forward(q, k, v, o, mask="causal"), "scored": lambda o: m.sdpa_scored_forward(q, k, v, o),
            "scored_lse": lambda o: m.sdpa_scored_forward_lse(q, k, v, o, lse)[0],
            "mha": lambda o: m.mha_forward(x, x, *w, 2, o, ws),
            "paged": lambda o: m.sdpa_paged_forward(pq, *c.args, c.row_starts, c.seq_lens, o, ws, mask="causal")}


@pytest.mark.parametrize("name", ["forward", "scored", "scored_lse", "mha", "paged"])
def test_a_threads_first_call(lib, name):
    call = calls(lib)[name]
    want = call(None)
    got, faults = torch.full_like(want, float("nan")), []
    torch.cuda.synchronize()

    def run():
        try:
            call(got)
        except Exception as e:  # noqa: BLE001
            faults.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join(60)
    assert not t.is_alive() and not faults, faults
    torch.cuda.synchronize()
    assert torch.equal(got, want)
