"""Gradients under slopes where a query sees far keys alone: every bias is large and only differences count."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import BF, gen, ints, lib, make, run  # noqa: E402,F401


@pytest.mark.parametrize("cap", [None, 20.0])
@pytest.mark.parametrize("slope", [0.5, -0.25])
@pytest.mark.parametrize("mask", ["key_padding", "causal_key_padding"])
def test_weights_of_a_row_keep_their_ratios(lib, cap, slope, mask):
    """One-hot output gradients lay single rows of P into dv: P_ij / P_il against the definition, at distances up to two
    million.  P and dv are rounded to bf16 once each, so a ratio is off by 4 U at most, beside the scores' own error (2^-18
    of the products' magnitudes, the cap's, a last rounding of the exponent)."""
    T_q, n = 1 << 21, 70
    g = gen(91)
    q = torch.zeros(1, 1, T_q, 64, device="cuda", dtype=BF)
    rows = [n + 5, 4000, 70_000, 1_000_003, T_q - 129, T_q - 1]
    q[0, 0, rows] = torch.randn(len(rows), 64, generator=g, device="cuda").to(BF)
    k, v = (torch.randn(1, 1, 100, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    go = torch.zeros_like(q)
    for x, r in enumerate(rows):
        go[0, 0, r, x] = 1.0
    form = {"mask": mask, "key_lens": ints(n), "slopes": torch.tensor([slope], device="cuda"), "cap": cap}
    lo = torch.empty_like(q)
    o, lse = lib.sdpa_scored_forward_lse(q, k, v, out_lo=lo, **form)
    dv = lib.sdpa_scored_backward(q, k, v, o, go, lse, o_lo=lo, **form)[2][0, 0, :n].double()
    for x, r in enumerate(rows):
        z = q[0, 0, r].double() @ k[0, 0, :n].double().t() * 0.125
        mag = (q[0, 0, r].double().abs() @ k[0, 0, :n].double().abs().t() * 0.125).max().item()
        s = cap * torch.tanh(z / cap) if cap else z
        p = torch.softmax(s - slope * (r - torch.arange(n, device="cuda", dtype=torch.float64)), 0)
        top = int(p.argmax())
        keep = p > 1e-9
        ratio, want = dv[keep, x] / dv[top, x], p[keep] / p[top]
        tol = 4.1 * ref.U + 2 * (2.0 ** -18 * mag + 2.0 ** -15 + (6e-4 if cap else 0.0))
        off = (ratio / want - 1).abs().max().item()
        assert off <= tol, (r, off, tol)
        # the factor they share: the fp32 lse's rounding, and 2 U of the largest
        total = abs(torch.log(dv[top, x] / p[top]).item())
        assert total <= 2.0 ** -22 * abs(lse[0, 0, r].item()) + 2.1 * ref.U + 2 * tol, (r, total)


@pytest.mark.parametrize("cap", [None, 20.0])
@pytest.mark.parametrize("slopes", [[0.5, 0.03], [-0.2, 0.5]])
def test_gradients_against_the_definition(lib, cap, slopes, monkeypatch):
    """Rows up to 3,000 past 70 keys, with a bound on a score that does not grow with its bias: products, cap, and the lse's
    rounding, which stands for e^(2^-22 |lse|) in P."""
    q, k, v, go = make(1, 2, 2, 3000, 3000, 92)
    form = {"mask": "key_padding", "key_lens": ints(70), "cap": cap, "slopes": torch.tensor(slopes, device="cuda")}
    mag = (q.double().abs() @ k[:, :, :70].double().abs().transpose(2, 3) * 0.125).max()
    most = 2.0 ** -22 * (0.5 * 3000 + 40)
    monkeypatch.setattr(ref, "score_error", lambda c, s: torch.zeros_like(s) + 2.0 ** -18 * mag + most + 2.0 ** -20 + (6e-4 if c else 0.0))
    want = ref.attention(q, k, v, scale=0.125, dout=go, **form)
    got = run(lib, q, k, v, go, form)
    for n in ("o", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n], want[n + "_tol"], 0)


@pytest.mark.parametrize("T_q,T_k,mask", [(700, 700, "none"), (700, 700, "causal"), (90, 600, "none"), (600, 90, "none"),
                                          (300, 300, "prefix")])
@pytest.mark.parametrize("cap", [None, 20.0])
def test_columns_on_both_sides_of_the_diagonal(lib, T_q, T_k, mask, cap):
    """Blocks of keys before, across and past the queries, steep and rising biases."""
    q, k, v, go = make(2, 4, 2, T_q, T_k, 93)
    form = {"mask": mask, "cap": cap, "slopes": torch.tensor([0.7, -0.05, 0.01, 3.0], device="cuda")}
    if mask == "prefix":
        form.update(mask="causal", prefix_lens=ints(140, 30))
    want = ref.attention(q, k, v, scale=0.125, dout=go, **form)
    got = run(lib, q, k, v, go, form)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n], want[n + "_tol"], 0)
