"""Cases of the paged K/V cache: writing it, reading it back, and the attention of new tokens over it.

    write    each sequence's new rows of K and V go into their pages; an int8 cache is read back with them
    read     the cached rows of every sequence as contiguous bf16
    attend   each sequence's new tokens (a prompt, a chunk of one, drafted tokens, a single token) over its cached rows

Heads have 64 features, as in the library's attention calls; new rows and queries are bf16, packed (heads, tokens, 64);
pages (pages, K/V heads, rows, 64) are bf16, or int8 with one power of two for each row.  With `own` false run() computes
the operators from elementary torch operations in fp32, rounded once at the end; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

HD = 64
BF = torch.bfloat16


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # two long prompts into an empty cache
        _case("write_prompts_bf16_2x8192", "write", B=2, h=16, page=64, ctx=(0, 0), new=(8192, 8192)),
        # one generated token for each of sixteen requests: the call's own latency
        _case("write_step_bf16_16", "write", B=16, h=16, page=16, ctx=(100, 1023), new=(1, 1)),
        # a ragged batch of prompts, quantised, and read back
        _case("write_prompts_int8_16x512", "write", B=16, h=8, page=32, int8=True, ctx=(0, 0), new=(100, 512)),
        # one token and a few drafted ones behind short contexts, quantised, and read back
        _case("write_drafts_int8_8", "write", B=8, h=8, page=16, int8=True, ctx=(1, 200), new=(1, 5), token_major=True),
        # quantised caches of sixteen requests handed to a call that takes contiguous ones
        _case("read_int8_16x8192", "read", B=16, h=16, page=64, int8=True, ctx=(4096, 8192)),
        # one short request
        _case("read_bf16_1000", "read", B=1, h=8, page=16, ctx=(1000, 1000)),
        # two whole prompts of the library's headline length
        _case("attend_prompts_bf16_2x8192", "attend", B=2, h=16, page=64, ctx=(0, 0), new=(8192, 8192)),
        # a chunk of a prompt behind a long quantised context, four query heads on each K/V head
        _case("attend_chunk_int8_1024_behind_32768", "attend", B=1, h=16, h_kv=4, page=64, int8=True, ctx=(31744, 31744),
              new=(1024, 1024), token_major=True),
        # an odd chunk of one request among the single tokens of others
        _case("attend_mixed_bf16_33", "attend", B=33, h=16, h_kv=4, page=32, ctx=(500, 4000), new=(1, 1), first=777),
        # the library's decoding workload, from pages
        _case("attend_step_bf16_16x8192", "attend", B=16, h=16, page=64, ctx=(4095, 8191), new=(1, 1)),
        # many requests on a quantised cache, eight query heads on each K/V head
        _case("attend_step_int8_64x8192", "attend", B=64, h=16, h_kv=2, page=16, int8=True, ctx=(4095, 8191), new=(1, 1),
              token_major=True),
        # one short request
        _case("attend_step_bf16_1x100", "attend", B=1, h=8, page=16, ctx=(100, 100), new=(1, 1)),
    ]


def _case(name, op, **kw):
    """ctx: cached rows before the new ones, from and to; new: new rows of a sequence, from and to; first: new rows of the
    first sequence, if others than those; page: rows of a page."""
    c = {"op": op, "B": 1, "h": 8, "h_kv": 0, "page": 16, "int8": False, "first": 0, "causal": True, "token_major": False,
         "new": (0, 0)}
    c.update(kw)
    c["h_kv"] = c["h_kv"] or c["h"]
    c["ctx_lo"], c["ctx_hi"] = c.pop("ctx")
    c["new_lo"], c["new_hi"] = c.pop("new")
    if name:
        c["name"] = name
    return c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# what a drawn case has at most: rows of 64 in the cache, (query, key) pairs over all heads
_MOST_ROWS, _MOST_PAIRS = 1 << 21, 1 << 30


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    kw = {"page": rng.choice([16, 32, 48, 64, 128, 256]), "int8": rng.random() < 0.5, "token_major": rng.random() < 0.5}
    g = rng.choice([1, 1, 2, 3, 4, 8]) if op == "attend" else 1
    h_kv = rng.choice([1, 2, 3, 4, 8, 16])
    kind = rng.choice(["prompts", "chunks", "drafts", "step", "step", "mixed"])
    if op == "read":
        ctx, new = _log_int(rng, 16, 32768), 0
    elif kind == "prompts":
        ctx, new = 0, _log_int(rng, 16, 8192)
    elif kind == "chunks":
        ctx, new = _log_int(rng, 16, 32768), _log_int(rng, 16, 2048)
    elif kind == "drafts":
        ctx, new = _log_int(rng, 16, 32768), rng.randint(2, 8)
    else:
        ctx, new = _log_int(rng, 16, 32768), 1
    first = _log_int(rng, 16, 1024) if kind == "mixed" and op != "read" else 0
    rows = h_kv * (ctx + max(new, first))
    pairs = h_kv * g * max(new, 1) * (ctx + new) + h_kv * g * first * (ctx + first)
    while h_kv > 1 and (rows > _MOST_ROWS or pairs > _MOST_PAIRS):
        h_kv, rows, pairs = h_kv // 2, rows // 2, pairs // 2
    most = max(1, min(64, _MOST_ROWS // max(rows, 1), _MOST_PAIRS // max(pairs, 1)))
    kw.update(B=_log_int(rng, 1, most), h=h_kv * g, h_kv=h_kv, first=first)
    kw["ctx"] = (ctx // 2, ctx)
    kw["new"] = (max(1, new // 2), new) if new else (0, 0)
    kw["causal"] = op != "attend" or rng.random() < 0.8
    return _case(None, op, **kw)


# ------------------------------------------------------------------------------------------------------- inputs
def _power(e):
    """2^e in fp32, -126 <= e <= 127."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x):
    """(whole numbers in fp32, exponents) of rows x (..., 64): the least exponent e >= -126 under which the row fits into
    -127 2^e .. 127 2^e, and the row in steps of 2^e, halves to even."""
    x = x.float()
    mantissa, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(mantissa <= 127.0 / 128.0, e - 7, e - 6).clamp(min=-126).to(torch.int32)
    return torch.round(x * _power(-e)[..., None]), e


def _lengths(case):
    """(new rows, rows cached before them) of every sequence, spread evenly over their ranges; a seed gives their order."""
    c = case

    def spread(lo, hi):
        x = [lo + (hi - lo) * (2 * i + 1) // (2 * c["B"]) for i in range(c["B"])]
        random.Random(c["B"]).shuffle(x)
        return x

    new, ctx = spread(c["new_lo"], c["new_hi"]), spread(c["ctx_lo"], c["ctx_hi"])[::-1]
    if c["first"]:
        new[0] = c["first"]
    return list(zip(new, ctx))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    pick = random.Random(seed)
    c = case
    B, h, hk, P = c["B"], c["h"], c["h_kv"], c["page"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def packed(heads, tokens):  # as a projection leaves it, token by token or head by head
        if c["token_major"]:
            return normal(tokens, heads, HD).to(BF).transpose(0, 1)
        return normal(heads, tokens, HD).to(BF)

    pairs = _lengths(c)
    rest = pairs[1:] if c["first"] else pairs
    pick.shuffle(rest)
    pairs = pairs[:len(pairs) - len(rest)] + rest
    new, lens = [n for n, _ in pairs], [n + before for n, before in pairs]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    used = [(n + P - 1) // P for n in lens]
    pages = sum(used) + 7  # some that no sequence holds
    order = list(range(pages))
    pick.shuffle(order)
    table, at = [], 0
    for u in used:
        table.append(order[at:at + u] + [-1] * (max(used) - u))
        at += u

    def whole(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    st = {"case": c, "new": new, "lens": lens, "starts": starts, "page_table": whole(table), "row_starts": whole(starts),
          "seq_lens": whole(lens), "max_new": max(new), "rows": max(lens), "scale": 1.0 / math.sqrt(HD),
          "k_scales": None, "v_scales": None}
    for name in ("k", "v"):
        # every page holds what was cached before: rows of differing sizes, as normalised and rotated heads have them
        x = (normal(pages, hk, P, HD) * torch.exp(0.5 * normal(pages, hk, P, 1))).to(BF)
        if c["int8"]:
            n, e = _quantise(x)
            st[name + "_pages"], st[name + "_scales"] = n.to(torch.int8), (e + 127).to(torch.uint8)
        else:
            st[name + "_pages"] = x
    if c["op"] == "write":
        st["k"], st["v"] = packed(hk, starts[-1]), packed(hk, starts[-1])
    elif c["op"] == "attend":
        st["q"] = packed(h, starts[-1])
    return st


# ---------------------------------------------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[state["case"]["op"]](state)


def _run_own(st):
    import transformer_scaled_dot_softmax_gb300 as mha

    c = st["case"]
    cache = (st["k_pages"], st["v_pages"], st["page_table"])
    scales = {"k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    if c["op"] == "attend":
        return mha.sdpa_paged_forward(st["q"], *cache, st["row_starts"], st["seq_lens"], max_new=st["max_new"],
                                      scale=st["scale"], mask="causal" if c["causal"] else "none", **scales)
    if c["op"] == "write":
        mha.paged_cache_append(st["k"], st["v"], *cache, st["row_starts"], st["seq_lens"], **scales)
        if not c["int8"]:
            return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    k, v = mha.paged_cache_read(*cache, st["seq_lens"], rows=st["rows"], **scales)
    return {"k": k, "v": v}


def _plain_write(st):
    c, dev = st["case"], st["k"].device
    token = torch.arange(st["starts"][-1], device=dev)
    b = torch.searchsorted(st["row_starts"][1:].contiguous(), token, right=True)
    pos = (st["seq_lens"] - st["row_starts"][1:])[b] + token
    page, at = st["page_table"][b, pos // c["page"]].long(), pos % c["page"]
    for name in ("k", "v"):
        x = st[name].transpose(0, 1)  # (tokens, heads, 64)
        if c["int8"]:
            x, e = _quantise(x)
            st[name + "_scales"][page, :, at] = (e + 127).to(torch.uint8)
        st[name + "_pages"][page, :, at] = x.to(st[name + "_pages"].dtype)
    if not c["int8"]:
        return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    return _plain_read(st)


def _rows_of(st, name, pages):
    """Cached rows (..., heads, rows, 64) of a list of pages (..., n), in fp32."""
    x = st[name + "_pages"][pages].float()
    if st["case"]["int8"]:
        x = x * _power(st[name + "_scales"][pages].int() - 127)[..., None]
    x = x.movedim(-4, -3)  # (..., heads, n, page rows, 64)
    return x.reshape(*x.shape[:-3], -1, HD)


def _plain_read(st):
    c, dev = st["case"], st["page_table"].device
    pages = st["page_table"].long().clamp(min=0)
    there = torch.arange(st["rows"], device=dev) < st["seq_lens"][:, None]
    out = {}
    for name in ("k", "v"):
        x = _rows_of(st, name, pages)[:, :, :st["rows"]]
        out[name] = torch.where(there[:, None, :, None], x, 0.0).to(BF)
    return out


def _plain_attend(st):
    c, q = st["case"], st["q"]
    hk, g = c["h_kv"], c["h"] // c["h_kv"]
    out = torch.empty_like(q)
    for b in range(c["B"]):
        n, length = st["new"][b], st["lens"][b]
        rows = slice(st["starts"][b], st["starts"][b + 1])
        pages = st["page_table"][b, :(length + c["page"] - 1) // c["page"]].long()
        k, v = _rows_of(st, "k", pages)[:, :length], _rows_of(st, "v", pages)[:, :length]
        s = q[:, rows].float().reshape(hk, g * n, HD) @ k.transpose(1, 2) * st["scale"]
        if c["causal"] and n > 1:
            pos = torch.arange(length - n, length, device=q.device).repeat(g)
            s.masked_fill_(torch.arange(length, device=q.device) > pos[:, None], -math.inf)
        s = torch.exp(s.sub_(s.amax(-1, keepdim=True)))
        out[:, rows] = (s @ v / s.sum(-1, keepdim=True)).reshape(hk * g, n, HD).to(BF)
    return out


# --------------------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    row = HD + 1 if c["int8"] else 2 * HD  # a cached row's bytes
    lengths, heads = _lengths(c), c["h_kv"]
    tokens, cached = sum(n for n, _ in lengths), sum(n + before for n, before in lengths)
    written = 2 * heads * tokens * (2 * HD + row)
    back = 2 * heads * cached * (row + 2 * HD)
    if c["op"] == "read":
        return {"bytes": back, "flops": 0.0}
    if c["op"] == "write":
        return {"bytes": written + (back if c["int8"] else 0), "flops": 0.0}
    pairs = sum(n * before + (n * (n + 1) // 2 if c["causal"] else n * n) for n, before in lengths)
    return {"bytes": 2 * heads * cached * row + 2 * c["h"] * tokens * 2 * HD, "flops": 4.0 * HD * c["h"] * pairs}


# -------------------------------------------------------------------------------------------------------- exact
def _exact_cached(st, name, pages, head):
    """Cached rows of several pages, end to end, fp64."""
    x = st[name + "_pages"][pages, head].double()
    if st["case"]["int8"]:
        x = x * torch.exp2(st[name + "_scales"][pages, head].double() - 127.0)[:, :, None]
    return x.reshape(-1, HD)


def _exact_stored(x):
    """The values that an int8 cache holds for rows x (rows, 64)."""
    x = x.double()
    top = x.abs().max(1).values
    step = torch.full_like(top, 2.0 ** -126)
    need = torch.ceil(torch.log2(torch.clamp(top, min=1e-45) / 127.0)) - 1  # or one more, two more: by comparison
    for more in range(4):
        candidate = torch.exp2(torch.clamp(need + more, min=-126.0))
        step = torch.where((top <= 127.0 * step), step, candidate)
    down = torch.floor(x / step[:, None])
    rest = x / step[:, None] - down
    up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(down, 2.0) == 1.0))
    return (down + up) * step[:, None]


def exact(case, seed):
    c, st = case, prepare(case, seed)
    P, hk, B = c["page"], c["h_kv"], c["B"]
    g, table = c["h"] // hk, st["page_table"].tolist()
    if c["op"] == "attend":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
        for b in range(B):
            n, length = st["new"][b], st["lens"][b]
            pages = torch.tensor(table[b][:-(-length // P)], device=out.device)
            limit = torch.arange(n, device=out.device)[:, None] + (length - n)
            seen = torch.arange(length, device=out.device)[None, :] <= (limit if c["causal"] else length)
            for a in range(hk):
                k, v = (_exact_cached(st, name, pages, a)[:length] for name in ("k", "v"))
                for i in range(a * g, (a + 1) * g):
                    s = st["q"][i, st["starts"][b]:st["starts"][b + 1]].double() @ k.t() * st["scale"]
                    w = torch.softmax(torch.where(seen, s, -math.inf), 1)
                    out[i, st["starts"][b]:st["starts"][b + 1]] = w @ v
        return out
    if c["op"] == "write" and not c["int8"]:
        out = {name: st[name].double() for name in ("k_pages", "v_pages")}
        for b in range(B):
            for t in range(st["new"][b]):
                p = st["lens"][b] - st["new"][b] + t
                for name in ("k", "v"):
                    out[name + "_pages"][table[b][p // P], :, p % P] = st[name][:, st["starts"][b] + t].double()
        return out
    out = {}
    for name in ("k", "v"):
        x = torch.zeros((B, hk, st["rows"], HD), dtype=torch.float64, device="cuda")
        for b in range(B):
            length = st["lens"][b]
            pages = torch.tensor(table[b][:-(-length // P)], device="cuda")
            for a in range(hk):
                x[b, a, :length] = _exact_cached(st, name, pages, a)[:length]
                if c["op"] == "write":
                    rows = slice(st["starts"][b], st["starts"][b + 1])
                    x[b, a, length - st["new"][b]:length] = _exact_stored(st[name][a, rows])
        out[name] = x
    return out
