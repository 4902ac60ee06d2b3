"""More work items for each processor than its on-chip item table holds (128), most of them without a key, in every form of
the forward and of decoding: past the table a warp computes its items one by one, and those without keys pass no barrier
between the warp's lanes but the item's own."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import BF, bias_args, gen, lib, make  # noqa: E402,F401


@pytest.mark.parametrize("bias,cap", [("none", None), ("slopes", None), ("buckets", 10.0)])
@pytest.mark.parametrize("B,h", [(160, 150), (700, 40)])  # ranked by length in the kernel, and not
def test_forward(lib, bias, cap, B, h):
    q, k, v, _ = make(B, h, h // 5, 3, 3, 101)
    lens = torch.randint(-1, 4, (B,), generator=gen(102), device="cuda", dtype=torch.int32)
    lens[torch.rand(B, generator=gen(103), device="cuda") < 0.6] = 0
    form = {"mask": "causal_key_padding", "key_lens": lens, "cap": cap, **bias_args(bias, h, 104)}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = ref.attention(q, k, v, scale=0.125, **form)
    fine = ref.attention(q, k, v, scale=0.125, two_parts=True, **form)
    for _ in range(3):
        o = torch.full_like(q, float("nan"))
        lib.sdpa_scored_forward(q, k, v, o, status=status, **form)
        o2, lse = lib.sdpa_scored_forward_lse(q, k, v, torch.full_like(q, float("nan")), status=status, **form)
        assert int(status.item()) == 0
        ref.check("o", o, want["o"], want["o_tol"], 0)
        ref.check("o2", o2, fine["o"], fine["o_tol"], 0)
        ref.check("lse", lse, want["lse"], want["lse_tol"], 0)
        assert torch.all(o[lens <= 0] == 0) and torch.all(lse[lens <= 0] == -float("inf"))


@pytest.mark.parametrize("bias,cap", [("none", None), ("slopes", 10.0), ("buckets", None)])
@pytest.mark.parametrize("P", [0, 5])
def test_decoding(lib, bias, cap, P):
    B, h, T_q, T_k = 1400, 16, 2, 5
    g = gen(105)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    x = [n(B, h, T_q, 64), n(h, P, 64), n(h, P, 64), n(B, h, T_k, 64), n(B, h, T_k, 64)]
    lens = torch.randint(0, T_k + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[torch.rand(B, generator=gen(106), device="cuda") < 0.7] = 0
    form = {"cap": cap, **bias_args(bias, h, 107)}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, tol = ref.decode(*x, lens, scale=0.125, **form)
    for _ in range(3):
        o = torch.full_like(x[0], float("nan"))
        lib.sdpa_decode_shared_forward(*x, lens, o, status=status, **form)
        assert int(status.item()) == 0
        ref.check("o", o, want, tol, 0)
        if P == 0:
            assert torch.all(o[lens == 0] == 0)
