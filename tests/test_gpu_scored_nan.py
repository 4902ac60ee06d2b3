"""NaN and infinities among the scores that a query sees: they reach its output, its log-sum-exp and the gradients, and no
other query's; a query that sees none of them keeps its values."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_scored import bias_args, gen, ints, lib, make, run  # noqa: E402,F401

BF = torch.bfloat16
NAN = float("nan")


def all_nan(t):
    return bool(torch.isnan(t.float()).all())


def keeps(name, got, want, rows):
    """The rows' values are the definition's."""
    ref.check(name, got[:, :, rows], want[name][:, :, rows], want[name + "_tol"][:, :, rows], 0)


@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
@pytest.mark.parametrize("cap", [None, 20.0])
@pytest.mark.parametrize("at", [0, 63, 200, 399])
def test_in_one_query(lib, bias, cap, at):
    T = 400
    q, k, v, go = make(2, 4, 2, T, T, 81)
    form = {"mask": "causal", "cap": cap, **bias_args(bias, 4, 82)}
    want = ref.attention(q, k, v, scale=0.125, dout=go, **form)
    q[:, :, at, 5] = NAN
    got = run(lib, q, k, v, go, form)
    rest = [i for i in range(T) if i != at]
    for n in ("o", "o2", "lse"):
        assert all_nan(got[n][:, :, at]), n
        keeps(n.replace("o2", "o"), got[n], want, rest)
    keeps("dq", got["dq"], want, rest)
    assert all_nan(got["dq"][:, :, at])
    for n in ("dk", "dv"):
        assert all_nan(got[n][:, :, : at + 1]), n
    # blocks of keys past the query see nothing of it
    past = [j for j in range(T) if j // 128 > at // 128]
    for n in ("dk", "dv"):
        if past:
            keeps(n, got[n], want, past)
    if bias == "buckets":
        assert bool(torch.isnan(got["dtable"].float()).any())


@pytest.mark.parametrize("bias", ["none", "slopes", "buckets"])
@pytest.mark.parametrize("cap", [None, 20.0])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_in_one_key(lib, bias, cap, value):
    """Key 150: the causal queries from there on see it.  (+infinity uncapped, times features of either sign, is NaN or an
    infinite score; capped, it is NaN or the cap.)"""
    T, at = 300, 150
    q, k, v, go = make(2, 4, 2, T, T, 83)
    q[..., 7] = q[..., 7].abs().clamp(min=0.01)
    form = {"mask": "causal", "cap": cap, **bias_args(bias, 4, 84)}
    want = ref.attention(q, k, v, scale=0.125, **form)
    k[:, :, at, 7] = value
    got = run(lib, q, k, v, go, form)
    if value != value or not cap:
        for n in ("o", "o2", "lse"):
            assert all_nan(got[n][:, :, at:]), n
        assert all_nan(got["dq"][:, :, at:])
    else:  # tanh(inf) = 1: a finite score
        for n in ("o", "o2", "lse"):
            assert bool(torch.isfinite(got[n]).all()), n
    for n in ("o", "o2", "lse"):
        keeps(n.replace("o2", "o"), got[n], want, list(range(at)))


@pytest.mark.parametrize("cap", [None, 20.0])
def test_in_every_key(lib, cap):
    q, k, v, go = make(1, 2, 2, 140, 140, 85)
    k.fill_(NAN)
    got = run(lib, q, k, v, go, {"mask": "key_padding", "key_lens": ints(135), "cap": cap})
    for n in ("o", "o2", "lse", "dq"):
        assert all_nan(got[n]), n
    assert all_nan(got["dv"][:, :, :135])
    # and a batch entry that sees no key is still 0
    q, k, v, go = make(2, 2, 2, 140, 140, 86)
    k.fill_(NAN)
    got = run(lib, q, k, v, go, {"mask": "key_padding", "key_lens": ints(0, 140), "cap": cap})
    assert torch.all(got["o"][0] == 0) and torch.all(got["lse"][0] == -float("inf")) and torch.all(got["dq"][0] == 0)
    assert all_nan(got["o"][1])


def test_negative_infinity_is_no_weight(lib):
    """A visible score of -infinity: the key has weight 0, the others theirs."""
    T, at = 200, 70
    q, k, v, go = make(1, 2, 2, T, T, 87)
    q[..., 3] = 1.0
    k[..., 3] = 0.0
    k2 = torch.cat((k[:, :, :at], k[:, :, at + 1:]), 2).contiguous()
    v2 = torch.cat((v[:, :, :at], v[:, :, at + 1:]), 2).contiguous()
    want = ref.attention(q, k2, v2, scale=0.125)
    k[:, :, at, 3] = -float("inf")
    o, lse = lib.sdpa_scored_forward_lse(q, k, v)
    ref.check("o", o, want["o"], want["o_tol"], 0)
    ref.check("lse", lse, want["lse"], want["lse_tol"], 0)


def caches(B, h, h_kv, T_q, P, T_k, seed):
    g = gen(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    return [n(B, h, T_q, 64), n(h_kv, P, 64), n(h_kv, P, 64), n(B, h_kv, T_k, 64), n(B, h_kv, T_k, 64)]


@pytest.mark.parametrize("h_kv,T_q", [(4, 1), (2, 1), (4, 3)])
@pytest.mark.parametrize("cap", [None, 20.0])
@pytest.mark.parametrize("P", [0, 700])
def test_decoding(lib, h_kv, T_q, cap, P):
    """In one request's cache (first, middle, last row, every row of a cache of one), in one query row, in the prefix."""
    B, T_k = 6, 300
    lens = ints(300, 300, max(T_q, 1), 250, 300, 120)
    form = {"cap": cap, **bias_args("slopes", 4, 0)}
    x = caches(B, 4, h_kv, T_q, P, T_k, 88)
    want, tol = ref.decode(*x, lens, scale=0.125, **form)
    x[3][0, :, 0] = NAN      # first row
    x[3][1, :, 299] = NAN    # last row
    x[3][2, :, : int(lens[2])] = NAN  # every row that counts
    x[3][3, :, 137, 9] = NAN
    x[3][5, :, 120:] = NAN   # past the length
    x[0][4, 1] = NAN         # one head's queries
    got = lib.sdpa_decode_shared_forward(*x, lens, **form)
    for b in range(4):
        assert all_nan(got[b]), b
    assert all_nan(got[4, 1])
    for b, heads in ((4, [0, 2, 3]), (5, [0, 1, 2, 3])):
        ref.check("o", got[b, heads], want[b, heads], tol[b, heads], 0)
    if P:
        x = caches(B, 4, h_kv, T_q, P, T_k, 88)
        x[1][0, 650, 2] = NAN  # K/V head 0's prefix: its query heads, in every request
        got = lib.sdpa_decode_shared_forward(*x, lens, **form)
        own = 4 // h_kv
        assert all_nan(got[:, :own])
        ref.check("o", got[:, own:], want[:, own:], tol[:, own:], 0)


def test_decoding_of_one_key(lib):
    for P, T_k in ((0, 1), (1, 0), (1, 1)):
        x = caches(2, 2, 2, 1, P, T_k, 89)
        for t in (x[1], x[3]):
            t.fill_(NAN)
        assert all_nan(lib.sdpa_decode_shared_forward(*x))
    x = caches(2, 2, 2, 1, 0, 5, 90)
    x[3].fill_(NAN)
    o = lib.sdpa_decode_shared_forward(*x, ints(0, 1))
    assert torch.all(o[0] == 0) and all_nan(o[1])
