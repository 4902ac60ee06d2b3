"""The contiguous forwards over so many keys that a query block's key tiles are summed in several runs (as
test_gpu_paged_runs.py's)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import scored_reference as ref  # noqa: E402
from test_gpu_paged_runs import TILES  # noqa: E402
from test_gpu_scored_windows import SCALE, forms, keys, rows  # noqa: E402
from test_gpu_scored import BF, gen, ints, lib, run  # noqa: E402,F401

PAGE = 1 << 16


@pytest.mark.parametrize("copies,lens", [(1, None), (4, None), (5, 4 * PAGE + 1), (17, 16 * PAGE + 777), (64, None)])
def test_values_of_one_sign_over_many_keys(lib, copies, lens):
    """65,536 keys over and over, with padding past the length: the average of values between 0.5 and 1."""
    g = gen(71)
    k, v = torch.randn(PAGE, 64, generator=g, device="cuda").to(BF), (torch.rand(PAGE, 64, generator=g, device="cuda") / 2 + 0.5).to(BF)
    q = torch.randn(1, 1, 300, 64, generator=g, device="cuda").to(BF)
    T, n = copies * PAGE, lens or copies * PAGE
    kk, vv = (x.repeat(copies, 1).reshape(1, 1, T, 64) for x in (k, v))
    s = q[0, 0].double() @ k.double().t() * 0.125
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - top) * (n // PAGE + (torch.arange(PAGE, device="cuda") < n % PAGE))
    lse = torch.log(w.sum(-1)) + top[:, 0]
    want = (w / w.sum(-1, keepdim=True)) @ v.double()
    e = 2 * ref.score_error(None, 0.125 * (q[0, 0].double().abs() @ k.double().abs().t())).amax(-1, keepdim=True)
    tol = (ref.U + e) * 2 * want + ref.U * want
    pad = {} if lens is None else {"mask": "key_padding", "key_lens": ints(n)}
    ref.check("plain", lib.sdpa_forward(q, kk, vv, **pad)[0, 0], want, tol, 0)
    o, l = lib.sdpa_forward_lse(q, kk, vv, **pad)
    ref.check("plain, with lse", o[0, 0], want, tol, 0)
    ref.check("its lse", l[0, 0], lse, ref.U + e[:, 0], 0)  # of rounded weights
    kk[:, :, n:], vv[:, :, n:] = float("nan"), float("nan")  # (the scored forward clears them)
    slopes = torch.zeros(1, device="cuda")
    for form in ({}, {"cap": 50.0}, {"slopes": slopes}):
        c = form.get("cap")
        z = c * torch.tanh(s / c) if c else s
        w = torch.exp(z - z.amax(-1, keepdim=True)) * (n // PAGE + (torch.arange(PAGE, device="cuda") < n % PAGE))
        a, b = (w / w.sum(-1, keepdim=True)) @ v.double(), torch.log(w.sum(-1)) + z.amax(-1)
        x = 2 * ref.score_error(c, 0.125 * (q[0, 0].double().abs() @ k.double().abs().t())).amax(-1, keepdim=True)
        ref.check("scored", lib.sdpa_scored_forward(q, kk, vv, **pad, **form)[0, 0], a, (ref.U + x) * 2 * a + ref.U * a, 0)
        o, l = lib.sdpa_scored_forward_lse(q, kk, vv, **pad, **form)
        # weights in two parts: the bias alone would show at a sixteenth of this
        ref.check("scored, with lse", o[0, 0], a, (ref.U ** 2 + x + 2.0 ** -12) * 2 * a + ref.U * a, 0)
        ref.check("scored lse", l[0, 0], b, x[:, 0] + 2.0 ** -22 * b.abs(), 0)


@pytest.mark.parametrize("name", list(TILES))
@pytest.mark.parametrize("form", ["plain", "cap", "buckets"])
def test_references_that_differ_between_runs(lib, name, form):
    """Both directions, in documents of all keys: gradients take the log-sum-exp of every run."""
    g = gen(72)
    k, v = keys(TILES[name], g, (1, 1))
    q, go = rows(g, 1, 2, 70), torch.randn(1, 2, 70, 64, generator=g, device="cuda").to(BF)
    form = {"scale": SCALE, **forms(2)[form]}
    got = run(lib, q, k, v, go, form)
    want, fine = ref.attention(q, k, v, dout=go, **form), ref.attention(q, k, v, two_parts=True, **form)
    ref.check("o2", got["o2"], fine["o"], fine["o_tol"], 0)
    for n, m in (("o", "o"), ("lse", "lse"), ("dq", "dq"), ("dk", "dk"), ("dv", "dv")):
        ref.check(n, got[n], want[m], want[m + "_tol"], 0)
    if len(form) > 1:
        return
    # the plain forward holds sums of 2^-64 to 2^16: here its first step is exact
    o, l = lib.sdpa_forward_lse(q, *(x.expand(1, 2, -1, -1).contiguous() for x in (k, v)), scale=SCALE)
    ref.check("plain", o, want["o"], want["o_tol"], 0)
    ref.check("plain lse", l, want["lse"], ref.U + want["lse_tol"], 0)
    ref.check("plain", lib.sdpa_forward(q, *(x.expand(1, 2, -1, -1).contiguous() for x in (k, v)), scale=SCALE), want["o"],
              want["o_tol"], 0)


@pytest.mark.parametrize("B,h,T_q", [(1, 1, 1), (2, 3, 1), (1, 2, 3)])
def test_decoding_over_a_long_prefix(lib, B, h, T_q):
    """A prefix of 2^21 rows of one sign, and caches."""
    g = gen(73)
    k, v = torch.randn(h, PAGE, 64, generator=g, device="cuda").to(BF), (torch.rand(h, PAGE, 64, generator=g, device="cuda") / 2 + 0.5).to(BF)
    q = torch.randn(B, h, T_q, 64, generator=g, device="cuda").to(BF)
    cache = [torch.zeros(B, h, 10, 64, dtype=BF, device="cuda") for _ in "kv"]
    out = lib.sdpa_decode_shared_forward(q, k.repeat(1, 32, 1), v.repeat(1, 32, 1), *cache, ints(*[0] * B))
    s = q.double() @ k.double().transpose(1, 2) * 0.125
    want = torch.softmax(s, -1) @ v.double()
    e = 2 * ref.score_error(None, 0.125 * (q.double().abs() @ k.double().abs().transpose(1, 2))).amax(-1, keepdim=True)
    ref.check("o", out, want, (ref.U + e) * 2 * want + ref.U * want, 0)


@pytest.mark.parametrize("form", ["plain", "causal", "slopes", "buckets", "documents", "prefix", "padded"])
def test_masks_and_biases_over_many_keys(lib, form):
    """300,000 queries and keys: rows on both sides of the ends of documents, prefixes, lengths and runs."""
    T, dev = 300_000, "cuda"
    g = gen(74)
    q, k, v = (torch.randn(1, 1, T, 64, generator=g, device=dev).to(BF) for _ in range(3))
    i = torch.tensor([0, 127, 128, 9_999, 10_000, 131_071, 131_072, 141_500, 262_143, 262_144, 273_000, T - 129, T - 1], device=dev)
    j = torch.arange(T, device=dev)
    kw, vis = {"mask": "causal"}, j[None] <= i[:, None]
    bias = torch.zeros(len(i), T, dtype=torch.float64, device=dev)
    if form == "slopes":
        kw["slopes"] = torch.tensor([2.0 ** -14], device=dev)
        bias = -(2.0 ** -14) * (j[None] - i[:, None]).abs().double()
    elif form == "buckets":
        starts = (0, 1, 300, 20_000)
        kw["table"], kw["bucket_starts"] = torch.randn(4, 1, generator=g, device=dev).to(BF), starts
        bias = ref.bias_of(j[None] - i[:, None], 1, None, kw["table"], starts)[0]
    elif form == "documents":
        ids = (j >= 10_000).int() + (j >= 273_000).int()
        kw["doc_ids"] = ids[None].contiguous()
        vis = vis & (ids[None] == ids[i][:, None])
    elif form == "prefix":
        kw["prefix_lens"] = ints(141_500)
        vis = vis | (j[None] < 141_500)
    elif form == "padded":
        kw = {"mask": "key_padding", "key_lens": ints(299_001)}
        vis = (j[None] < 299_001).expand(len(i), -1)
    x = q[0, 0, i].double()
    p, _, lse, s = ref.weights(x @ k[0, 0].double().t() * 0.125, None, bias, vis)
    mag = 0.125 * (x.abs() @ k[0, 0].double().abs().t()) + bias.abs()
    e = 2 * torch.where(vis, ref.score_error(None, mag), 0.0).amax(-1, keepdim=True)
    want = p @ v[0, 0].double()
    spread = p @ v[0, 0].double().abs() + want.abs()
    tol = (ref.U + e) * spread + ref.U * want.abs()
    if form in ("plain", "padded"):
        o, l = lib.sdpa_forward_lse(q, k, v, **kw)
        ref.check("o", o[0, 0, i], want, tol, 0)
        ref.check("lse", l[0, 0, i], lse, ref.U + e[:, 0], 0)
        ref.check("o", lib.sdpa_forward(q, k, v, **kw)[0, 0, i], want, tol, 0)
    if form != "plain":
        ref.check("o", lib.sdpa_scored_forward(q, k, v, **kw)[0, 0, i], want, tol, 0)
        lo = torch.empty_like(q)
        o, l = lib.sdpa_scored_forward_lse(q, k, v, out_lo=lo, **kw)
        ref.check("o", o[0, 0, i], want, tol, 0)
        ref.check("lse", l[0, 0, i], lse, e[:, 0] + 2.0 ** -22 * lse.abs(), 0)
        # with what rounding took from it: the weights' second parts, and runs' sums (2^-12)
        both = o[0, 0, i].double() + lo[0, 0, i].double()
        ref.check("o + lo", both, want, (ref.U ** 2 + e + 2.0 ** -12) * spread + ref.U ** 2 * want.abs(), 0)
