"""Scored attention on the host: refusals of the C entry points before anything is launched, workspace sizes, bucket
borders; and the fp64 reference of the GPU tests against torch's autograd."""
import ctypes
import math

import pytest

FAKE = 1 << 20  # never dereferenced: every case fails its checks first


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from transformer_scaled_dot_softmax_gb300 import _native
    return _native


def form(lib, cap=0.0, slopes=None, table=None, starts=None, n=None, both=0, prefix=None, docs=None):
    f = lib.ScoreForm()
    f.cap, f.slopes, f.table, f.bidirectional, f.prefix_lens, f.doc_ids = cap, slopes, table, both, prefix, docs
    f.num_buckets = n if n is not None else len(starts) if starts else 0
    if starts:
        f._keep = (ctypes.c_int32 * len(starts))(*starts)
        f.bucket_starts = ctypes.addressof(f._keep)
    return f


def fwd(lib, f=None, dt=1, p=FAKE, k=FAKE, lse=None, lo=None, ws=FAKE, ws_bytes=1 << 40, B=1, h=2, hk=2, Tq=8, Tk=8, d=64, scale=0.125,
        mask=0, lens=None):
    return lib.lib.sdpa_scored_forward(dt, p, k, k, p, lse, lo, ws, ws_bytes, B, h, hk, Tq, Tk, d, d, scale, mask, lens,
                                       None if f is None else ctypes.addressof(f), None, None)


def bwd(lib, f=None, dt=1, p=FAKE, lse=FAKE, dtable=None, ws=FAKE, ws_bytes=1 << 40, B=1, h=2, hk=2, Tq=8, Tk=8, d=64,
        scale=0.125, mask=0, lens=None):
    return lib.lib.sdpa_scored_backward(dt, p, p, p, p, None, p, lse, p, p, p, dtable, ws, ws_bytes, B, h, hk, Tq, Tk, d, d, scale,
                                        mask, lens, None if f is None else ctypes.addressof(f), None, None)


def dec(lib, f=None, p=FAKE, kp=FAKE, ws=FAKE, ws_bytes=1 << 40, B=1, h=2, hk=2, Tq=1, Tp=8, Tk=8, d=64, scale=0.125, mask=0,
        lens=None):
    return lib.lib.sdpa_decode_shared_forward(p, kp, kp, p, p, p, ws, ws_bytes, B, h, hk, Tq, Tp, Tk, d, d, scale, mask, lens,
                                              None if f is None else ctypes.addressof(f), None, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    bad, uns = lib.MHA_ERR_INVALID_ARG, lib.MHA_ERR_UNSUPPORTED
    assert call(lib, p=None) == bad
    assert call(lib, B=-1) == bad and call(lib, Tk=-1) == bad and call(lib, hk=0) == bad
    assert call(lib, h=3, hk=2) == bad                                   # heads do not divide
    assert call(lib, dt=7) == bad and call(lib, dt=0) == uns
    assert call(lib, d=128) == uns and call(lib, d=0) == bad
    assert call(lib, scale=float("nan")) == bad and call(lib, mask=4) == bad
    assert call(lib, mask=2) == bad                                      # key padding without lengths
    assert call(lib, Tq=1 << 24) == uns
    assert call(lib, p=FAKE + 8) == lib.MHA_ERR_MISALIGNED
    assert call(lib, B=0) == lib.MHA_OK and call(lib, h=0, hk=0) == lib.MHA_OK
    for f in (form(lib, cap=-1.0), form(lib, cap=float("nan")), form(lib, cap=float("inf")), form(lib, cap=1e-45),
              form(lib, slopes=FAKE, table=FAKE, starts=(0, 1)), form(lib, table=FAKE), form(lib, starts=(0, 1)),
              form(lib, table=FAKE, starts=(1, 2)), form(lib, table=FAKE, starts=(0, 2, 2)), form(lib, table=FAKE, n=4),
              form(lib, table=FAKE, starts=(0,), n=-1), form(lib, prefix=FAKE)):
        assert call(lib, f) == bad
    assert call(lib, form(lib, docs=FAKE), Tq=4) == bad                  # documents need T_q == T_k
    assert call(lib, form(lib, table=FAKE, starts=tuple(range(65)))) == uns
    assert call(lib, form(lib, table=FAKE, starts=(0, 65537))) == uns
    for f in (form(lib, table=FAKE, starts=(0, 1)), form(lib, docs=FAKE)):
        assert call(lib, f, ws=None) == lib.MHA_ERR_WORKSPACE
        assert call(lib, f, ws_bytes=8) == lib.MHA_ERR_WORKSPACE
        assert call(lib, f, ws=FAKE + 16) == lib.MHA_ERR_MISALIGNED


def test_the_remainder_needs_the_log_sum_exp(lib):
    assert fwd(lib, lo=FAKE) == lib.MHA_ERR_INVALID_ARG
    assert fwd(lib, lse=FAKE, lo=FAKE + 2) == lib.MHA_ERR_MISALIGNED


def test_backward_refusals(lib):
    assert bwd(lib, lse=None) == lib.MHA_ERR_INVALID_ARG
    assert bwd(lib, dtable=FAKE) == lib.MHA_ERR_INVALID_ARG              # a gradient of no table
    assert bwd(lib, ws=None) == lib.MHA_ERR_WORKSPACE
    assert bwd(lib, Tq=0, Tk=0) == lib.MHA_OK


def test_decode_refusals(lib):
    bad = lib.MHA_ERR_INVALID_ARG
    assert dec(lib, p=None) == bad and dec(lib, kp=None) == bad
    assert dec(lib, Tp=-1) == bad and dec(lib, h=3) == bad and dec(lib, mask=2) == bad and dec(lib, mask=9) == bad
    assert dec(lib, Tq=9) == lib.MHA_ERR_UNSUPPORTED and dec(lib, d=32) == lib.MHA_ERR_UNSUPPORTED
    assert dec(lib, Tp=1 << 24) == lib.MHA_ERR_UNSUPPORTED
    assert dec(lib, form(lib, prefix=FAKE), mask=1) == bad and dec(lib, form(lib, docs=FAKE)) == bad
    assert dec(lib, p=FAKE + 2) == lib.MHA_ERR_MISALIGNED and dec(lib, kp=FAKE + 8) == lib.MHA_ERR_MISALIGNED
    assert dec(lib, ws=None) == lib.MHA_ERR_WORKSPACE and dec(lib, ws_bytes=512) == lib.MHA_ERR_WORKSPACE
    assert dec(lib, ws=FAKE + 128) == lib.MHA_ERR_MISALIGNED
    assert dec(lib, B=0) == lib.MHA_OK and dec(lib, Tq=0) == lib.MHA_OK


def test_workspace_sizes(lib):
    r = lambda x: (x + 255) // 256 * 256  # noqa: E731
    f = lambda *a: lib.lib.sdpa_scored_workspace_bytes(*a[:4], ctypes.addressof(a[4]) if a[4] else None)  # noqa: E731
    assert f(2, 3, 130, 7, None) == 0 and f(-1, 3, 1, 1, None) == 0
    t = form(lib, table=FAKE, starts=(0, 100))
    assert f(2, 3, 130, 7, t) == r(3 * (2 * 368 + 16) * 4)        # distances past 100 + 256 and padding
    assert f(2, 3, 7, 7, form(lib, docs=FAKE)) == r(2 * 7 * 8)
    assert f(2, 3, 7, 7, form(lib, table=FAKE, starts=(0, 0))) == 0
    b = lib.lib.sdpa_scored_backward_workspace_bytes
    plain = 256 + 2 * 3 * 256 * 64 * 4 + 2 * 2 * 3 * 256 * 4  # the item counter's 256 bytes, dQ's sums, two row terms
    assert b(2, 3, 3, 130, 7, None) == plain and b(2, 3, 2, 130, 7, None) == 0
    # three query heads on one K/V head, a CTA and fp32 sums of dk and dv each
    assert b(2, 3, 1, 130, 7, None) == plain + 2 * r(3 * 2 * 1 * 7 * 64 * 4)
    # the expanded bias and one sum per head, key block and bucket
    assert b(2, 3, 3, 130, 7, ctypes.addressof(t)) == plain + r(3 * (2 * 368 + 16) * 4) + r(2 * 368 + 16) + r(2 * 3 * 1 * 2 * 4)
    d = lib.lib.sdpa_decode_shared_workspace_bytes
    assert d(4, 8, 2, 1, 0, 0, None) == 0 and d(4, 8, 3, 1, 10, 10, None) == 0
    assert d(4, 8, 2, 1, 100, 0, None) == 4 * 8 * 256 + r(4 * 8 * 8)     # one key range of the prefix
    assert d(4, 8, 2, 1, 100, 90, None) == 2 * 4 * 8 * 256 + r(2 * 4 * 8 * 8)


def test_relative_bucket_starts():
    import transformer_scaled_dot_softmax_gb300 as m
    starts = m.relative_bucket_starts(32, 128)
    assert starts[:17] == tuple(range(17)) and len(starts) == 32
    for n, far in ((32, 128), (16, 128), (8, 777), (2, 2), (64, 4096)):
        starts = m.relative_bucket_starts(n, far)
        assert starts[0] == 0 and all(a < b for a, b in zip(starts, starts[1:])) and starts[-1] <= far
    # 8 exact buckets, then half an octave each: the borders that are powers of two are exact
    starts = m.relative_bucket_starts(16, 128)
    assert [starts[i] for i in (8, 10, 12, 14)] == [8, 16, 32, 64]
    assert starts[9] == math.ceil(8 * 2 ** 0.5)
    for args in ((1, 10), (16, 8)):
        with pytest.raises(ValueError):
            m.relative_bucket_starts(*args)


@pytest.mark.parametrize("cap", [None, 3.0])
@pytest.mark.parametrize("bias", ["none", "slopes", "table"])
def test_reference_against_autograd(cap, bias):
    torch = pytest.importorskip("torch")
    import scored_reference as ref
    g = torch.Generator().manual_seed(1)
    B, h, hk, T = 2, 4, 2, 23
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, go = n(B, h, T, 64), n(B, hk, T, 64), n(B, hk, T, 64), n(B, h, T, 64)
    starts = (0, 1, 2, 5)
    slopes = torch.tensor([0.5, 0.1, 0.0, -0.2], dtype=torch.float64) if bias == "slopes" else None
    table = n(8, h) if bias == "table" else None
    ids = torch.cumsum((torch.rand(B, T, generator=g) < 0.2).int(), 1)
    lens, pre = torch.tensor([23, 11]), torch.tensor([4, 0])
    leaves = [x.clone().requires_grad_() for x in (q, k, v) + ((table,) if table is not None else ())]
    d = torch.arange(T)[None] - torch.arange(T)[:, None]
    b = 0.0
    if slopes is not None:
        b = -slopes[:, None, None] * d.abs()
    if table is not None:
        idx = torch.tensor([[sum(abs(int(x)) >= s for s in starts) - 1 + (4 if x > 0 else 0) for x in r] for r in d])
        b = leaves[3][idx].permute(2, 0, 1)
    z = leaves[0] @ leaves[1].repeat_interleave(2, 1).transpose(2, 3) * 0.125
    s = (cap * torch.tanh(z / cap) if cap else z) + b
    vis = torch.zeros(B, 1, T, T, dtype=torch.bool)
    for x in range(B):
        for i in range(T):
            for j in range(T):
                vis[x, 0, i, j] = j < lens[x] and (j <= i or j < pre[x]) and ids[x, i] == ids[x, j]
    p = torch.softmax(s.masked_fill(~vis, -math.inf), -1)
    p = torch.where(vis.any(-1, keepdim=True), p, 0.0)
    o = torch.nan_to_num(p) @ leaves[2].repeat_interleave(2, 1)
    got = ref.attention(q, k, v, scale=0.125, cap=cap, slopes=slopes, table=table, bucket_starts=starts,
                        mask="causal_key_padding", key_lens=lens, prefix_lens=pre, doc_ids=ids, dout=go)
    assert torch.allclose(got["o"], o, atol=1e-12)
    seen = vis.any(-1).expand(B, h, T)
    (o * go)[seen].sum().backward()
    for name, x in zip(("dq", "dk", "dv", "dtable"), leaves):
        assert torch.allclose(got[name], torch.nan_to_num(x.grad), atol=1e-10), name
