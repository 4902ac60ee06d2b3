"""Capped scores over the whole range of caps: the error that a score may have does not grow with the cap."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import gen, ints, lib, make, run  # noqa: E402,F401

BF = torch.bfloat16
CAPS = [1e-18, 1e-9, 1e-3, 0.5, 50.0, 60.0, 100.0, 500.0, 1000.0, 5000.0, 1e5, 1e6, 1e9, 1e13, 1e18]


def score_error(cap, s_abs):
    """What include/mha.h grants a capped score (6e-4, 2^-20 of itself), and fp32 products and sums of 64 terms."""
    return 6e-4 + (2.0 ** -20 + 2.0 ** -18) * s_abs + 2.0 ** -20


def attention(q, k, v, go, form):
    """scored_reference's values and bounds with that error in its scores', and 1 - t^2 (off by 1.7e-5 in the polynomials'
    range, of which the reference counts 6e-6)."""
    old = ref.score_error
    ref.score_error = score_error
    try:
        r = ref.attention(q, k, v, scale=0.125, dout=go, **form)
        fine = ref.attention(q, k, v, scale=0.125, two_parts=True, **form)
    finally:
        ref.score_error = old
    g = q.shape[1] // k.shape[1]
    qq, go = q.double(), go.double()
    ke, ve = (x.double().repeat_interleave(g, 1) for x in (k, v))
    vis = ref.visible(q.shape[0], q.shape[2], k.shape[2], q.device, form.get("mask", "none"))[:, None]
    bias = ref.bias_of(torch.arange(k.shape[2], device="cuda")[None] - torch.arange(q.shape[2], device="cuda")[:, None],
                       q.shape[1], form.get("slopes"), None, None)
    p = ref.weights(qq @ ke.transpose(2, 3) * 0.125, form["cap"], bias, vis)[0]
    ds = 1.2e-5 * (p * (go @ ve.transpose(2, 3) - (go * r["o"]).sum(-1, keepdim=True))).abs()
    r["dq_tol"] += 0.125 * (ds @ ke.abs())
    r["dk_tol"] += 0.125 * (ds.transpose(2, 3) @ qq.abs()).reshape(k.shape[0], k.shape[1], g, *k.shape[2:]).sum(2)
    return r, fine


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("gain", [0.0, 3.0, 40.0])
@pytest.mark.parametrize("slopes", [False, True])
def test_forward_and_gradients(lib, cap, gain, slopes):
    q, k, v, go = make(2, 4, 2, 333, 333, 71, gain=gain)
    form = {"mask": "causal", "cap": cap}
    if slopes:
        form["slopes"] = torch.tensor([0.5, 0.1, 0.02, 0.0], device="cuda")
    got = run(lib, q, k, v, go, form)
    want, fine = attention(q, k, v, go, form)
    ref.check("o", got["o"], want["o"], want["o_tol"], 0)
    ref.check("o2", got["o2"], fine["o"], fine["o_tol"], 0)
    ref.check("lse", got["lse"], want["lse"], want["lse_tol"], 0)
    for n in ("dq", "dk", "dv"):
        ref.check(n, got[n], want[n], want[n + "_tol"], 0)


def one_feature(T, most):
    """q and k whose products are single, so that a score is exact before its cap: from -most to most."""
    q = torch.zeros(1, 1, T, 64, dtype=BF, device="cuda")
    k = torch.zeros(1, 1, T, 64, dtype=BF, device="cuda")
    q[..., 0] = 8.0
    k[0, 0, :, 0] = torch.linspace(-most, most, T, device="cuda").to(BF)
    return q, k


@pytest.mark.parametrize("cap", [c for c in CAPS if c >= 50])
@pytest.mark.parametrize("most", [1.0, 26.0, 100.0, 500.0, 5000.0])
def test_log_sum_exp_of_exact_scores(lib, cap, most):
    """Row i of a causal mask over rising scores: lse is the cap's value at its own key, and a little."""
    T = 520
    q, k = one_feature(T, most)
    v = torch.randn(1, 1, T, 64, generator=gen(72), device="cuda").to(BF)
    _, lse = lib.sdpa_scored_forward_lse(q, k, v, mask="causal", cap=cap)
    z = k[0, 0, :, 0].double()
    s = cap * torch.tanh(z / cap)
    want = torch.stack([torch.logsumexp(s[: i + 1], 0) for i in range(T)])
    # the score's granted error, lse's own fp32 roundings (log2 units, natural ones)
    tol = 6e-4 + 2.0 ** -20 * s.abs().cummax(0)[0] + 2.0 ** -21 * want.abs() + 2.0 ** -18
    off = (lse[0, 0].double() - want).abs()
    assert (off <= tol).all(), (off / tol).max().item()


@pytest.mark.parametrize("cap", [0.5, 60.0, 1000.0, 1e6, 1e9, 1e18])
@pytest.mark.parametrize("h_kv,T_q", [(4, 1), (2, 1), (4, 3)])
def test_decoding(lib, cap, h_kv, T_q):
    g = gen(73)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    B, h, P, T_k = 3, 4, 300, 200
    x = [(n(B, h, T_q, 64) * 4).to(BF)] + [n(*s).to(BF) for s in ((h_kv, P, 64), (h_kv, P, 64), (B, h_kv, T_k, 64), (B, h_kv, T_k, 64))]
    lens = ints(T_k, T_q, 77)
    old = ref.score_error
    ref.score_error = score_error
    try:
        want, tol = ref.decode(*x, lens, scale=0.125, cap=cap, mask="causal")
    finally:
        ref.score_error = old
    ref.check("o", lib.sdpa_decode_shared_forward(*x, lens, mask="causal", cap=cap), want, tol, 0)
