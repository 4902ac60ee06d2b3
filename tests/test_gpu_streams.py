"""Calls on a stream that is not the current one (stream=), without outputs or a workspace of the caller's, while the
current stream's work allocates and fills memory of the same sizes before and after them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF = torch.bfloat16
CYCLES = 20_000_000  # about 10 ms


@pytest.fixture(scope="module")
def lib():
    import transformer_scaled_dot_softmax_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def calls(m):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def n(*s, gain=1.0):
        return (torch.randn(s, generator=g, device="cuda") * gain).to(BF)

    B, h, T, D = 2, 4, 300, 256
    q, k, v, go, x = n(B, h, T, 64), n(B, h, T, 64), n(B, h, T, 64), n(B, h, T, 64), n(B, T, D)
    w = [n(D, D, gain=D ** -0.5) for _ in range(4)]
    one, gamma, beta = n(B, h, 1, 64), n(D), n(D)
    enc = {"w_q": w[0], "w_k": w[1], "w_v": w[2], "w_o": w[3], "gamma1": gamma, "beta1": beta, "w1": n(D, 512, gain=D ** -0.5),
           "b1": n(512), "w2": n(512, D, gain=512 ** -0.5), "b2": n(D), "gamma2": gamma, "beta2": beta}
    ids = torch.arange(T, device="cuda", dtype=torch.int32).div(77, rounding_mode="floor").expand(B, T).contiguous()
    form = {"mask": "causal", "doc_ids": ids, "table": n(16, h), "bucket_starts": m.relative_bucket_starts(16, 128)}
    bias = {"table": form["table"], "bucket_starts": form["bucket_starts"]}
    o, lse = m.sdpa_forward_lse(q, k, v)
    so, slse = m.sdpa_scored_forward_lse(q, k[:, :2].contiguous(), v[:, :2].contiguous(), **form)
    k2, v2 = k[:, :2].contiguous(), v[:, :2].contiguous()
    prefix = n(h, 700, 64), n(h, 700, 64)
    prefix2 = n(2, 700, 64), n(2, 700, 64)
    host = [t.cpu().pin_memory() for t in (q, k, v)]
    return {
        "forward": lambda s: m.sdpa_forward(q, k, v, stream=s),
        "forward_lse": lambda s: m.sdpa_forward_lse(q, k, v, stream=s),
        "forward_host": lambda s: m.sdpa_forward_host(*host, stream=s),
        "backward": lambda s: m.sdpa_backward(q, k, v, o, go, lse, stream=s),
        "positions": lambda s: m.positional_encoding_add(x, stream=s),
        "encoder": lambda s: m.encoder_layer_forward(x, enc, h, stream=s),
        "decode": lambda s: m.sdpa_decode_forward(one, k, v, stream=s),
        "mha": lambda s: m.mha_forward(x, x, *w, h, stream=s),
        "mha_norm": lambda s: m.mha_forward_add_layernorm(x, x, *w, gamma, beta, h, stream=s),
        "scored": lambda s: m.sdpa_scored_forward(q, k2, v2, stream=s, **form),
        "scored_lse": lambda s: m.sdpa_scored_forward_lse(q, k2, v2, stream=s, **form),
        "scored_backward": lambda s: m.sdpa_scored_backward(q, k2, v2, so, go, slse, stream=s, **form),
        "decode_shared": lambda s: m.sdpa_decode_shared_forward(one, *prefix, k, v, stream=s, **bias),
        "decode_shared_heads": lambda s: m.sdpa_decode_shared_forward(one, *prefix2, k2, v2, stream=s, **bias),
    }


NAMES = ["forward", "forward_lse", "forward_host", "backward", "positions", "encoder", "decode", "mha", "mha_norm", "scored",
         "scored_lse", "scored_backward", "decode_shared", "decode_shared_heads"]


def as_list(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def same(a, b):
    """Equal bits, or (dq, whose key blocks are added in no fixed order) within one rounding of the whole."""
    return torch.equal(a, b) or (a.double() - b.double()).norm() <= 2.0 ** -8 * a.double().norm()


@pytest.fixture(scope="module")
def table(lib):
    made = calls(lib)
    torch.cuda.synchronize()
    return made


def sizes(want):
    """Bytes of blocks to fill: those of the results, and every power of two, for the scratch."""
    return sorted({t.numel() * t.element_size() for t in want} | {1 << e for e in range(10, 24)})


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_current_stream(lib, table, name):
    call = table[name]
    want = as_list(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    nbytes = sizes(want)
    for _ in range(3):
        # blocks that the current stream dropped with work on them still queued
        torch.cuda._sleep(CYCLES)
        for n in nbytes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        # the call waits behind a delay on its own stream
        with torch.cuda.stream(side):
            torch.cuda._sleep(2 * CYCLES)
        got = as_list(call(side))
        # memory that the call dropped, taken and filled at once
        for n in nbytes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, got)), name


@pytest.mark.parametrize("name", [n for n in NAMES if n != "forward_host"])
def test_results_dropped_on_the_current_stream(lib, table, name):
    """A result is read on the current stream and dropped before that read has run; the next call on the side stream may not
    have its memory."""
    call = table[name]
    want = as_list(call(None))
    torch.cuda.synchronize()
    side, copies = torch.cuda.Stream(), []
    for _ in range(3):
        got = as_list(call(side))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(CYCLES)
        copies.append([t.clone() for t in got])
        del got
        with torch.cuda.stream(side):
            for t in want:
                torch.empty_like(t).fill_(float("nan"))
    torch.cuda.synchronize()
    for got in copies:
        assert all(same(a, b) for a, b in zip(want, got)), name
