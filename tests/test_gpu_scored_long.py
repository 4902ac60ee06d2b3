"""Scored attention at its longest: up to the most keys a call takes, tensors past 4 GB, distances past a million."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import BF, gen, ints, lib  # noqa: E402,F401

CHUNK = 1 << 18


def normal(g, *shape):
    """bf16 normals, made piece by piece."""
    x = torch.empty(shape, dtype=BF, device="cuda")
    for part in x.view(-1).split(1 << 27):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return x


def exact(q, pos, parts, cap=None, slope=0.0, causal=False):
    """o and lse of query rows q (n, 64) at positions pos, and the sum of w |v|; parts: (first position, k, v) in turn."""
    n = q.shape[0]
    m = torch.full((n, 1), -float("inf"), dtype=torch.float64, device="cuda")
    l, o, a = torch.zeros_like(m), torch.zeros(n, 64, dtype=torch.float64, device="cuda"), torch.zeros(n, 64, dtype=torch.float64, device="cuda")
    for at, k, v in parts:
        for i in range(0, k.shape[0], CHUNK):
            kk, vv = k[i:i + CHUNK].double(), v[i:i + CHUNK].double()
            d = torch.arange(at + i, at + i + kk.shape[0], device="cuda", dtype=torch.float64)[None] - pos[:, None].double()
            s = q.double() @ kk.t() * 0.125
            s = (cap * torch.tanh(s / cap) if cap else s) - slope * d.abs()
            if causal:
                s = s.masked_fill(d > 0, -float("inf"))
            new = torch.maximum(m, s.amax(1, keepdim=True))
            w, f = torch.exp(s - torch.where(new.isfinite(), new, 0.0)), torch.exp(torch.where(m.isfinite(), m - new, -float("inf")))
            l, o, a, m = l * f + w.sum(1, keepdim=True), o * f + w @ vv, a * f + w @ vv.abs(), new
    return o / l, (m + l.log())[:, 0], a / l


def close(name, got, want, mag, keys):
    """Roundings of the weights and of the output, the scores' error (products below 40), fp32 sums over `keys` keys in
    steps of 16, each of half a rounding's length 2^-24 at most either way."""
    e = 2 * (2.0 ** -18 * 40 + 2.0 ** -20) + 2 * 2.0 ** -24 * keys / 16
    tol = (ref.U + e) * (mag + want.abs()) + ref.U * want.abs()
    off = ((got.double() - want).abs() / tol).max().item()
    assert off <= 1, (name, off)


@pytest.mark.parametrize("shift", [0.0, 1.0])
def test_forward_over_the_most_keys(lib, shift):
    T_k, T_q = 8_388_480, 130
    g = gen(111)
    q, k, v = normal(g, 1, 1, T_q, 64), normal(g, 1, 1, T_k, 64), normal(g, 1, 1, T_k, 64)
    if shift:
        v.add_(shift)  # sums that only grow
    o = lib.sdpa_scored_forward(q, k, v)
    o2, lse = lib.sdpa_scored_forward_lse(q, k, v)
    want, wl, mag = exact(q[0, 0], torch.zeros(T_q, device="cuda"), [(0, k[0, 0], v[0, 0])])
    close("o", o[0, 0], want, mag, T_k)
    close("o2", o2[0, 0], want, mag, T_k)
    assert ((lse[0, 0].double() - wl).abs() <= 2.0 ** -18 * 40 + 2.0 ** -24 * T_k / 64).all()


@pytest.mark.parametrize("cap", [None, 20.0])
def test_forward_past_four_gigabytes(lib, cap):
    B, h, T = 3, 24, 500_000  # K and V 4.6 GB each
    g = gen(112)
    k, v = normal(g, B, h, T, 64), normal(g, B, h, T, 64)
    q = normal(g, B, h, 2, 64)
    o = lib.sdpa_scored_forward(q, k, v, cap=cap, mask="key_padding", key_lens=ints(T, 130, T - 1))
    for b, a, n in ((0, 0, T), (1, 7, 130), (2, 23, T - 1)):
        want, _, mag = exact(q[b, a], torch.zeros(2, device="cuda"), [(0, k[b, a, :n], v[b, a, :n])], cap=cap)
        close("o", o[b, a], want, mag, n)


def test_gradients_over_long_sides(lib):
    """Two query rows over a million keys, and a million query rows over two keys."""
    g = gen(113)
    for T_q, T_k in ((2, 1_100_003), (1_100_003, 2)):
        q, k, v, go = normal(g, 1, 2, T_q, 64), normal(g, 1, 2, T_k, 64), normal(g, 1, 2, T_k, 64), normal(g, 1, 2, T_q, 64)
        lo = torch.empty_like(q)
        form = {"slopes": torch.tensor([1e-6, 0.0], device="cuda")}
        o, lse = lib.sdpa_scored_forward_lse(q, k, v, out_lo=lo, **form)
        dq, dk, dv, _ = lib.sdpa_scored_backward(q, k, v, o, go, lse, o_lo=lo, **form)
        for a in range(2):
            x, kk, vv, gg = (t[0, a].double() for t in (q, k, v, go))
            d = (torch.arange(T_k, device="cuda")[None] - torch.arange(T_q, device="cuda")[:, None]).double()
            p = torch.softmax(x @ kk.t() * 0.125 - form["slopes"][a].double() * d.abs(), 1)
            dp = gg @ vv.t()
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            e = 2 * (2.0 ** -18 * 40 + 2.0 ** -20) + 2.0 ** -22 * 20
            # dP and D in fp32, P and dS rounded once, sums in steps of 16 rows or 128 keys, the result rounded
            ds_tol = (ref.U + e) * ds.abs() + p * (2.0 ** -14 * (gg.abs() @ vv.abs().t()) + (p * dp.abs()).sum(1, keepdim=True) * (e + ref.U ** 2))
            for name, got, want, mag, tol, n in (
                    ("dq", dq, 0.125 * ds @ kk, 0.125 * ds.abs() @ kk.abs(), 0.125 * ds_tol @ kk.abs(), T_k / 16),
                    ("dk", dk, 0.125 * ds.t() @ x, 0.125 * ds.abs().t() @ x.abs(), 0.125 * ds_tol.t() @ x.abs(), T_q / 16),
                    ("dv", dv, p.t() @ gg, p.t() @ gg.abs(), (ref.U + e) * p.t() @ gg.abs(), T_q / 16)):
                off = ((got[0, a].double() - want).abs() / (1.05 * tol + 2.0 ** -23 * n * mag + ref.U * want.abs() + 1e-30)).max().item()
                assert off <= 1, (name, T_q, a, off)


@pytest.mark.parametrize("h,h_kv,T_q", [(1, 1, 1), (2, 1, 1), (2, 2, 3)])
def test_decoding_behind_a_long_prefix(lib, h, h_kv, T_q):
    B, P, T_k = 2, 2_000_001, 300
    g = gen(114)
    x = [normal(g, B, h, T_q, 64), normal(g, h_kv, P, 64), normal(g, h_kv, P, 64), normal(g, B, h_kv, T_k, 64), normal(g, B, h_kv, T_k, 64)]
    slopes = torch.tensor([1e-6, 2e-6][:h], device="cuda")
    lens = ints(300, 77)
    o = lib.sdpa_decode_shared_forward(*x, lens, slopes=slopes, mask="causal")
    for b, n in enumerate(lens.tolist()):
        pos = P + n - T_q + torch.arange(T_q, device="cuda")
        for a in range(h):
            z = a * h_kv // h
            want, _, mag = exact(x[0][b, a], pos, [(0, x[1][z], x[2][z]), (P, x[3][b, z, :n], x[4][b, z, :n])],
                                 slope=slopes[a].item(), causal=True)
            close("o", o[b, a], want, mag, P)


@pytest.mark.parametrize("T_q", [1, 2])
def test_decoding_over_caches_past_four_gigabytes(lib, T_q):
    B, h, T_k = 9, 16, 260_000  # 4.8 GB each
    g = gen(115)
    x = [normal(g, B, h, T_q, 64), normal(g, h, 1000, 64), normal(g, h, 1000, 64), normal(g, B, h, T_k, 64), normal(g, B, h, T_k, 64)]
    lens = ints(T_k, 5, T_k, 100_000, T_k - 1, 0, 17, T_k, T_k)
    o = lib.sdpa_decode_shared_forward(*x, lens)
    for b, a in ((0, 0), (1, 3), (3, 15), (5, 2), (8, 15)):
        n = int(lens[b])
        want, _, mag = exact(x[0][b, a], torch.zeros(T_q, device="cuda"), [(0, x[1][a], x[2][a]), (0, x[3][b, a, :n], x[4][b, a, :n])])
        close("o", o[b, a], want, mag, n + 1000)
