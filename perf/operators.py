"""Cases of the attention operators whose scores are more than a scaled dot product.

    forward   o of capped / distance-biased / document- or prefix-masked attention
    train     the same forward and its backward: o, dq, dk, dv (and dtable of a learned bucket bias)
    decode    one decoding step of a batch that shares a prefix

Every tensor is bf16 with heads of 64 features, as the library's attention calls take them.  With `own` false run()
computes the operators from elementary torch operations in fp32, rounded once at the end; with `own` true it calls
the library.
"""
import math

import torch

own = False

HD = 64
BF = torch.bfloat16


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a long causal prefill with capped scores: the library's headline size
        _case("forward_capped_causal_8192", "forward", B=2, h=16, T_q=8192, T_k=8192, mask="causal", cap=50.0, gain=4.0),
        # decoder self-attention of a batch of ordinary length with one slope per head
        _case("forward_slopes_causal_512", "forward", B=16, h=8, T_q=512, T_k=512, mask="causal", slopes=True),
        # prompts whose first part is read in both directions, four query heads on each K/V head, an odd length
        _case("forward_prefix_shared_heads_2000", "forward", B=4, h=16, h_kv=4, T_q=2000, T_k=2000, mask="causal", prefix=True),
        # one short request: the call's own latency
        _case("forward_small_64", "forward", B=1, h=8, T_q=64, T_k=64, mask="causal", cap=30.0, slopes=True, gain=4.0),
        # training on packed documents with capped scores
        _case("train_capped_documents_8192", "train", B=2, h=16, T_q=8192, T_k=8192, mask="causal", cap=50.0, docs=12, gain=4.0),
        # training with slopes on an odd, padded batch, three query heads on each K/V head
        _case("train_slopes_padded_1111", "train", B=3, h=6, h_kv=2, T_q=1111, T_k=1111, mask="causal_key_padding", slopes=True),
        # decoder training with a learned bucket bias
        _case("train_buckets_causal_4096", "train", B=2, h=16, T_q=4096, T_k=4096, mask="causal", buckets=32, far=128),
        # encoder training with a learned bucket bias in both directions, padded to 512
        _case("train_buckets_encoder_512", "train", B=16, h=8, T_q=512, T_k=512, mask="key_padding", buckets=16, far=128,
              both=True),
        # a small batch of short sentences
        _case("train_buckets_small_77", "train", B=2, h=8, T_q=77, T_k=77, mask="none", buckets=16, far=128, both=True),
        # many requests behind one long instruction, slopes
        _case("decode_slopes_64x8192", "decode", B=64, h=16, T_q=1, P=8192, T_k=1024, slopes=True),
        # eight query heads on each K/V head, a very long shared document, capped scores
        _case("decode_capped_shared_heads_16x32768", "decode", B=16, h=16, h_kv=2, T_q=1, P=32768, T_k=2048, cap=50.0, gain=4.0),
        # a few requests that check four drafted tokens each, short prefix, bucket bias
        _case("decode_small_4x1000", "decode", B=4, h=8, T_q=4, P=1000, T_k=64, mask="causal_key_padding", buckets=32, far=128),
    ]


def _case(name, op, **kw):
    c = {"op": op, "B": 1, "h": 8, "h_kv": 0, "T_q": 64, "T_k": 64, "P": 0, "mask": "none", "cap": 0.0, "slopes": False,
         "buckets": 0, "far": 0, "both": False, "prefix": False, "docs": 0, "gain": 1.0}
    if op == "decode":
        c["mask"] = "key_padding"
    c.update(kw)
    c["h_kv"] = c["h_kv"] or c["h"]
    if name:
        c["name"] = name
    return c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (query, key) pairs over all heads that a drawn case has at most: the work of the largest listed one
_MOST_PAIRS = {"forward": 1 << 30, "train": 1 << 28}


def draw(rng):
    op = rng.choice(["forward", "train", "decode"])
    kw = {"cap": rng.choice([0.0, 20.0, 30.0, 50.0])}
    kw["gain"] = rng.choice([2.0, 4.0, 6.0]) if kw["cap"] else 1.0
    bias = rng.choice(["none", "slopes", "buckets"])
    kw["slopes"] = bias == "slopes"
    if bias == "buckets":
        kw["buckets"] = rng.choice([8, 16, 32])
        kw["far"] = rng.choice([64, 128, 200, 777])
    g = rng.choice([1, 1, 2, 3, 4, 8])  # query heads on each K/V head
    if op == "decode":
        h_kv, T_q = _log_int(rng, 1, 16), rng.choice([1, 1, 1, 2, 3, 5, 8])
        P, T_k = _log_int(rng, 16, 65536), max(T_q, _log_int(rng, 8, 4096))
        most = max(1, min(128, (1 << 27) // (h_kv * g * T_q * (P + T_k)), (1 << 20) // (h_kv * T_k)))
        kw.update(B=_log_int(rng, 1, most), h_kv=h_kv, h=h_kv * g, T_q=T_q, P=P, T_k=T_k)
        kw["mask"] = rng.choice(["key_padding", "causal_key_padding"])
        return _case(None, op, **kw)
    T = _log_int(rng, 24, 8192 if op == "forward" else 5000)
    mask = rng.choice(["none", "causal", "causal", "key_padding", "causal_key_padding"])
    T_q = T if "causal" in mask or rng.random() < 0.7 else _log_int(rng, 24, 5000)
    h_kv = rng.choice([1, 2, 3, 4, 8])
    while h_kv > 1 and h_kv * g * T * T_q > _MOST_PAIRS[op]:
        h_kv //= 2
    most = max(1, min(32, _MOST_PAIRS[op] // (h_kv * g * T * T_q)))
    kw.update(B=_log_int(rng, 1, most), h_kv=h_kv, h=h_kv * g, T_q=T_q, T_k=T, mask=mask)
    kw["both"] = bias == "buckets" and "causal" not in mask
    if "causal" in mask and rng.random() < 0.4:
        kw["prefix"] = True
    elif T_q == T and rng.random() < 0.4:
        kw["docs"] = rng.randint(2, 16)
    return _case(None, op, **kw)


# ------------------------------------------------------------------------------------------------------- inputs
def _bucket_starts(n, far):
    """First distance of each of n buckets: one distance each for the nearer half, then logarithmically wider ones up
    to `far`, from which on all share the last; in whole numbers, so that no border hangs on a rounding."""
    near = n // 2
    starts, d = list(range(near)), near
    for u in range(n - near):
        while d ** (n - near) < near ** (n - near - u) * far ** u:
            d += 1
        starts.append(max(d, starts[-1] + 1))
    return tuple(starts)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = case

    def normal(*shape, gain=1.0):
        return (torch.randn(shape, generator=g, device=dev) * gain).to(BF)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device=dev, dtype=torch.int32)

    B, h, hk, T_q, T_k = c["B"], c["h"], c["h_kv"], c["T_q"], c["T_k"]
    st = {"case": c, "q": normal(B, h, T_q, HD, gain=c["gain"]), "k": normal(B, hk, T_k, HD), "v": normal(B, hk, T_k, HD),
          "scale": 1.0 / math.sqrt(HD), "cap": c["cap"] or None, "slopes": None, "table": None, "starts": None,
          "key_lens": None, "prefix_lens": None, "doc_ids": None}
    if c["slopes"]:  # the usual geometric slopes, 2^(-8 i / h)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32, device=dev)
    if c["buckets"]:
        st["starts"] = _bucket_starts(c["buckets"], c["far"])
        st["table"] = normal(c["buckets"] * (2 if c["both"] else 1), h)
    if c["op"] == "decode":
        st["k_prefix"], st["v_prefix"] = normal(hk, c["P"], HD), normal(hk, c["P"], HD)
        st["key_lens"] = whole(T_q, T_k, B)  # the new rows are in the cache already
        return st
    if "key_padding" in c["mask"]:
        st["key_lens"] = whole(T_k // 2, T_k, B)
    if c["prefix"]:
        st["prefix_lens"] = whole(0, T_k // 2, B)
    if c["docs"]:  # documents of random lengths, packed end to end
        cuts = torch.zeros((B, T_k), dtype=torch.int32, device=dev)
        cuts.scatter_(1, whole(1, T_k - 1, B, c["docs"] - 1).long(), 1)
        st["doc_ids"] = torch.cumsum(cuts, 1, dtype=torch.int32)
    if c["op"] == "train":
        st["dout"] = normal(B, h, T_q, HD)
    return st


# ---------------------------------------------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return _plain_decode(state) if state["case"]["op"] == "decode" else _plain(state)


def _run_own(st):
    import transformer_scaled_dot_softmax_gb300 as mha

    c = st["case"]
    form = {"scale": st["scale"], "cap": st["cap"], "slopes": st["slopes"], "table": st["table"],
            "bucket_starts": st["starts"], "mask": c["mask"]}
    if c["op"] == "decode":
        return mha.sdpa_decode_shared_forward(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["key_lens"], **form)
    form.update(key_lens=st["key_lens"], prefix_lens=st["prefix_lens"], doc_ids=st["doc_ids"])
    if c["op"] == "forward":
        return mha.sdpa_scored_forward(st["q"], st["k"], st["v"], **form)
    o_lo = torch.empty_like(st["q"])
    o, lse = mha.sdpa_scored_forward_lse(st["q"], st["k"], st["v"], out_lo=o_lo, **form)
    dq, dk, dv, dtable = mha.sdpa_scored_backward(st["q"], st["k"], st["v"], o, st["dout"], lse, o_lo=o_lo, **form)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}


def _bucket_of(dist, starts, both):
    """Bucket of key position minus query position."""
    s = torch.tensor(starts, device=dist.device)
    if both:
        return torch.searchsorted(s, dist.abs().contiguous(), right=True) - 1 + (dist > 0) * len(starts)
    return torch.searchsorted(s, (-dist).clamp(min=0).contiguous(), right=True) - 1


def _plain_scores(st, z, dist):
    """(scores, tanh) of products z (..., h, rows, keys); dist: key minus query position, of z's last two dimensions."""
    z = z * st["scale"]
    t = None
    if st["cap"]:
        t = torch.tanh(z / st["cap"])
        z = t * st["cap"]
    if st["slopes"] is not None:
        z = z - st["slopes"][:, None, None] * dist.abs().unsqueeze(-3)
    if st["table"] is not None:
        bucket = _bucket_of(dist, st["starts"], st["case"]["both"])
        b = st["table"].float()[bucket]  # (..., rows, keys, h)
        z = z + b.movedim(-1, -3)
    return z, t


def _diagonals(x):
    """Sums of x (h, T_q, T_k) over equal j - i, from -(T_q - 1) up, in fp64: with a row length of one more than
    their number, laying the rows out again one shorter moves each row by one."""
    h, T_q, T_k = x.shape
    n = T_q + T_k - 1
    y = torch.nn.functional.pad(x.flip(1), (0, T_q)).reshape(h, -1)[:, : T_q * n]
    return y.reshape(h, T_q, n).sum(1, dtype=torch.float64)


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, 1.0)


def _visible(st, dev):
    """(B or 1, 1, T_q, T_k) truth values."""
    c = st["case"]
    i, j = torch.arange(c["T_q"], device=dev)[:, None], torch.arange(c["T_k"], device=dev)[None, :]
    vis = torch.ones((1, 1, c["T_q"], c["T_k"]), dtype=torch.bool, device=dev)
    if "causal" in c["mask"]:
        vis = vis & (j <= i)
        if st["prefix_lens"] is not None:
            vis = vis | (j < st["prefix_lens"][:, None, None, None])
    if st["key_lens"] is not None:
        vis = vis & (j < st["key_lens"][:, None, None, None])
    if st["doc_ids"] is not None:
        vis = vis & (st["doc_ids"][:, None, :, None] == st["doc_ids"][:, None, None, :])
    return vis


def _plain(st):
    c, dev = st["case"], st["q"].device
    B, h, hk, T_q, T_k = c["B"], c["h"], c["h_kv"], c["T_q"], c["T_k"]
    rows = (B, hk, h // hk * T_q)
    q, k, v = st["q"].float().reshape(*rows, HD), st["k"].float(), st["v"].float()
    dist = torch.arange(T_k, device=dev)[None, :] - torch.arange(T_q, device=dev)[:, None]
    s, t = _plain_scores(st, (q @ k.transpose(2, 3)).reshape(B, h, T_q, T_k), dist)
    p = _softmax(s.masked_fill_(~_visible(st, dev), -math.inf))
    del s
    pr = p.reshape(*rows, T_k)
    o = (pr @ v).reshape(B, h, T_q, HD).to(BF)
    if c["op"] == "forward":
        return o
    g = st["dout"].float().reshape(*rows, HD)
    dv = pr.transpose(2, 3) @ g
    dp = (g @ v.transpose(2, 3)).reshape(B, h, T_q, T_k)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    del dp, p, pr
    dtable = None
    if st["table"] is not None:
        dd = torch.arange(-(T_q - 1), T_k, device=dev)
        dtable = torch.zeros(st["table"].shape, dtype=torch.float64, device=dev)
        dtable = dtable.index_add(0, _bucket_of(dd, st["starts"], c["both"]), _diagonals(ds.sum(0)).t()).to(BF)
    if t is not None:
        ds = ds * (1 - t * t)
    ds = ds.reshape(*rows, T_k) * st["scale"]
    dq = (ds @ k).reshape(B, h, T_q, HD)
    dk = ds.transpose(2, 3) @ q
    return {"o": o, "dq": dq.to(BF), "dk": dk.to(BF), "dv": dv.to(BF), "dtable": dtable}


def _plain_decode(st):
    c, dev = st["case"], st["q"].device
    B, h, hk, T_q, T_k, P = c["B"], c["h"], c["h_kv"], c["T_q"], c["T_k"], c["P"]
    g = h // hk
    q = st["q"].float().reshape(B, hk, g * T_q, HD)
    lens = st["key_lens"][:, None, None]
    t = torch.arange(T_q, device=dev)[None, :, None]
    pos = P + lens - T_q + t  # (B, T_q, 1)
    shared = (q.transpose(0, 1).reshape(hk, B * g * T_q, HD) @ st["k_prefix"].float().transpose(1, 2))
    shared = shared.reshape(hk, B, g * T_q, P).transpose(0, 1).reshape(B, h, T_q, P)
    sp, _ = _plain_scores(st, shared, torch.arange(P, device=dev) - pos)
    sc = (q @ st["k"].float().transpose(2, 3)).reshape(B, h, T_q, T_k)
    j = torch.arange(T_k, device=dev)
    sc, _ = _plain_scores(st, sc, P + j - pos)
    vis = j < (lens - T_q + 1 + t if "causal" in c["mask"] else lens)
    p = _softmax(torch.cat((sp, sc.masked_fill_(~vis[:, None], -math.inf)), -1))
    pp = p[..., :P].reshape(B, hk, g * T_q, P).transpose(0, 1).reshape(hk, B * g * T_q, P)
    o = (pp @ st["v_prefix"].float()).reshape(hk, B, g * T_q, HD).transpose(0, 1)
    o = o + p[..., P:].reshape(B, hk, g * T_q, T_k) @ st["v"].float()
    return o.reshape(B, h, T_q, HD).to(BF)


# --------------------------------------------------------------------------------------------------------- work
def _pairs(case):
    """Visible (query, key) pairs of one query head over the batch; lengths that are drawn count with their mean."""
    c = case
    T_q, T_k = c["T_q"], c["T_k"]
    keys = 0.75 * T_k if "key_padding" in c["mask"] else float(T_k)
    if "causal" in c["mask"]:
        full = min(T_q, keys)
        pairs = full * (full + 1) / 2 + max(0.0, T_q - full) * keys
        if c["prefix"]:  # a prefix of p adds p (p - 1) / 2 pairs, p uniform in [0, T_k / 2]
            pairs += (T_k / 2) ** 2 / 6
    else:
        pairs = T_q * keys
    if c["docs"]:  # pieces of a line cut at random: the squares of their lengths sum to 2 / (pieces + 1)
        pairs *= 2.0 / (c["docs"] + 1)
    return c["B"] * pairs


def work(case):
    c = case
    q, kv = c["B"] * c["h"] * c["T_q"] * HD * 2, c["B"] * c["h_kv"] * HD * 2
    if c["op"] == "decode":
        own_keys = c["B"] * (c["T_q"] + c["T_k"]) / 2
        return {"bytes": 2 * q + 2 * (c["P"] + own_keys) * c["h_kv"] * HD * 2,
                "flops": 4.0 * HD * c["h"] * c["T_q"] * (c["B"] * c["P"] + own_keys)}
    keys = 0.75 * c["T_k"] if "key_padding" in c["mask"] else c["T_k"]
    if c["op"] == "forward":
        return {"bytes": 2 * q + 2 * keys * kv, "flops": 4.0 * HD * c["h"] * _pairs(c)}
    # q, dout in; o, dq out; k, v in; dk, dv out.  Five products backward and two forward.
    return {"bytes": 4 * q + 2 * keys * kv + 2 * c["T_k"] * kv, "flops": 14.0 * HD * c["h"] * _pairs(c)}


# -------------------------------------------------------------------------------------------------------- exact
def _exact_bias(c, st, head, d):
    """Bias of the distances d (key minus query position), fp64."""
    if st["slopes"] is not None:
        return -st["slopes"][head].double() * d.abs().double()
    if st["table"] is None:
        return 0.0
    n, bucket = len(st["starts"]), torch.zeros_like(d)
    away = d.abs() if c["both"] else torch.where(d < 0, -d, 0)
    for u, start in enumerate(st["starts"]):
        bucket = torch.where(away >= start, u, bucket)
    if c["both"]:
        bucket = torch.where(d > 0, bucket + n, bucket)
    return st["table"][:, head].double()[bucket], bucket


def _exact_weights(c, st, head, q, k, d, vis):
    """(weights, tanh or None, bucket or None) of query rows q against keys k, fp64."""
    s, t, bucket = q @ k.t() * st["scale"], None, None
    if st["cap"]:
        t = torch.tanh(s / st["cap"])
        s = st["cap"] * t
    b = _exact_bias(c, st, head, d)
    if isinstance(b, tuple):
        b, bucket = b
    s = torch.where(vis, s + b, -math.inf)
    lse = torch.logsumexp(s, 1, keepdim=True)
    return torch.where(vis, torch.exp(s - torch.where(lse.isfinite(), lse, 0.0)), 0.0), t, bucket


def exact(case, seed):
    c, st = case, prepare(case, seed)
    dev = st["q"].device
    g, T_q, T_k, P = c["h"] // c["h_kv"], c["T_q"], c["T_k"], c["P"]
    f = {n: st[n].double() for n in ("q", "k", "v", "dout", "k_prefix", "v_prefix") if n in st}
    lens = [T_k] * c["B"] if st["key_lens"] is None else st["key_lens"].tolist()
    o = torch.zeros_like(f["q"])
    if c["op"] == "decode":
        for b in range(c["B"]):
            pos = P + lens[b] - T_q + torch.arange(T_q, device=dev)
            j = torch.arange(P + lens[b], device=dev)
            vis = j[None] <= pos[:, None] if "causal" in c["mask"] else torch.ones(T_q, len(j), dtype=torch.bool, device=dev)
            for a in range(c["h"]):
                kk = torch.cat((f["k_prefix"][a // g], f["k"][b, a // g, : lens[b]]))
                vv = torch.cat((f["v_prefix"][a // g], f["v"][b, a // g, : lens[b]]))
                o[b, a] = _exact_weights(c, st, a, f["q"][b, a], kk, j[None] - pos[:, None], vis)[0] @ vv
        return o
    i, j = torch.arange(T_q, device=dev)[:, None], torch.arange(T_k, device=dev)[None, :]
    dq, dk, dv = torch.zeros_like(f["q"]), torch.zeros_like(f["k"]), torch.zeros_like(f["v"])
    dtable = None if st["table"] is None else torch.zeros(st["table"].shape, dtype=torch.float64, device=dev)
    for b in range(c["B"]):
        vis = (j < lens[b]).expand(T_q, T_k)
        if "causal" in c["mask"]:
            vis = vis & ((j <= i) if st["prefix_lens"] is None else (j < torch.clamp(i + 1, min=int(st["prefix_lens"][b]))))
        if st["doc_ids"] is not None:
            vis = vis & (st["doc_ids"][b][:, None] == st["doc_ids"][b][None, :])
        for a in range(c["h"]):
            q, k, v = f["q"][b, a], f["k"][b, a // g], f["v"][b, a // g]
            w, t, bucket = _exact_weights(c, st, a, q, k, j - i, vis)
            o[b, a] = w @ v
            if c["op"] == "forward":
                continue
            do = f["dout"][b, a]
            dv[b, a // g] += w.t() @ do
            ds = w * (do @ v.t() - (do * o[b, a]).sum(1, keepdim=True))
            if dtable is not None:
                dtable[:, a] += torch.bincount(bucket.reshape(-1), ds.reshape(-1), len(dtable))
            if t is not None:
                ds = ds * (1 - t * t)
            dq[b, a] = st["scale"] * (ds @ k)
            dk[b, a // g] += st["scale"] * (ds.t() @ q)
    return o if c["op"] == "forward" else {"o": o, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}
