"""A paged K/V cache, its 8-bit rows and attention over it from the definition, on plain tensors and in fp64.

Bounds of attention, as scored_reference.py's: u = 2^-8 is one bf16 rounding; a weight enters P V after a score error and
rounded to bf16, numerator and normaliser with the same weights, so that o moves by at most (u + e)(sum w |v| + |o|), and is
rounded once, u |o|.  An int8 cache adds none: its values are bf16 numbers, and its products keep them whole.  (A query row
enters those products as fp16 numbers, at most 2^-39 of its largest element off: below the fp32 sums' error.)
Weights vanish below 2^-51 of their row's largest: a sum is kept against a reference that serves while a round's weights sum
to at most 2^64, over up to 2^10 rounds of a row here; when it moves, to leave a largest weight of at least 2^-1, a factor
below 2^-126 is flushed to 0, and with it at most 2^(64 + 10 - 126 + 1) of what remains, each part times a value.
"""
import math

import torch

import scored_reference as ref

BF = torch.bfloat16
U = ref.U


def stored(x):
    """(whole numbers, exponents + 127) of rows x (..., 64) by the definition, in fp64."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, 0.0)
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -126, dtype=torch.int64, device=x.device)
    for c in range(-126, 128):  # the least exponent that holds the row
        e = torch.where(top > 127.0 * torch.exp2(e.double()), torch.full_like(e, c + 1), e)
    n = torch.round(x * torch.exp2(-e.double())[..., None])  # halves to even
    n = torch.where((e == 122)[..., None], n.clamp(-63, 63), n)  # 2^128 is no bf16 number
    return n.to(torch.int8), torch.where(finite, e + 127, 255).to(torch.uint8)


def values(n, s):
    v = n.double() * torch.exp2(s.double() - 127.0)[..., None]
    return torch.where((s == 255)[..., None], math.nan, v)


class Cache:
    """B sequences of `lens` rows, the last `new` of which are new, in pages drawn at random from a pool whose other rows
    hold NaN (bf16), or anything with a NaN's exponent (int8)."""

    def __init__(self, h_kv, page, lens, new, int8=False, seed=0, capacity=0, spare=3, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.g, self.h_kv, self.page, self.int8, self.dev = g, h_kv, page, int8, device
        self.lens, self.new, self.B = list(lens), list(new), len(lens)
        used = [-(-n // page) for n in self.lens]
        self.max_pages = max(used + [-(-capacity // page)])
        self.pages = sum(used) + spare
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.page_table = table.to(device)
        starts = [0]
        for n in self.new:
            starts.append(starts[-1] + n)
        self.starts, self.N = starts, starts[-1]
        self.row_starts = torch.tensor(starts, dtype=torch.int32, device=device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        shape = (self.pages, h_kv, page, 64)
        self.k_scales = self.v_scales = None
        if int8:
            self.k_pages, self.v_pages = (torch.randint(-127, 128, shape, generator=g, device=device).to(torch.int8) for _ in "kv")
            self.k_scales, self.v_scales = (torch.full(shape[:3], 255, dtype=torch.uint8, device=device) for _ in "kv")
        else:
            self.k_pages, self.v_pages = (torch.full(shape, math.nan, dtype=BF, device=device) for _ in "kv")
        # every row of every sequence: k, v (h_kv, rows, 64) bf16
        self.rows = [tuple((self.normal(h_kv, n, 64) * torch.exp(0.5 * self.normal(h_kv, n, 1))).to(BF) for _ in "kv")
                     for n in self.lens]

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device=self.dev)

    @property
    def scales(self):
        return {"k_scales": self.k_scales, "v_scales": self.v_scales}

    @property
    def args(self):
        return self.k_pages, self.v_pages, self.page_table

    def put(self, b, first, last, rows=None):
        """Rows first .. last - 1 of a sequence into its pages, by plain indexing."""
        j = torch.arange(first, last, device=self.dev)
        pg, at = self.page_table[b].long()[j // self.page], j % self.page
        for i, name in enumerate("kv"):
            x = (self.rows[b] if rows is None else rows)[i][:, first:last].transpose(0, 1)
            if self.int8:
                n, s = stored(x)
                getattr(self, name + "_pages")[pg, :, at] = n
                getattr(self, name + "_scales")[pg, :, at] = s
            else:
                getattr(self, name + "_pages")[pg, :, at] = x

    def fill(self, new=True):
        for b, n in enumerate(self.lens):
            self.put(b, 0, n if new else n - self.new[b])
        return self

    def packed_new(self):
        """k, v (h_kv, N, 64) of all new rows."""
        return tuple(torch.cat([self.rows[b][i][:, self.lens[b] - n:] for b, n in enumerate(self.new)], 1) for i in range(2))

    def cached(self, b):
        """What the cache holds of a sequence's rows, fp64."""
        return tuple(values(*stored(x)) if self.int8 else x.double() for x in self.rows[b])


def attend(q, c, causal, scale=0.125, gone=None):
    """(o, bound) for packed queries (h, N, 64); gone[b]: truth values of the rows whose page is not there."""
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.full(q.shape, 1e-30, dtype=torch.float64, device=q.device)
    g = q.shape[0] // c.h_kv
    for b in range(c.B):
        n, length, rows = c.new[b], c.lens[b], slice(c.starts[b], c.starts[b + 1])
        if n == 0 or length == 0:
            continue
        k, v = (x.repeat_interleave(g, 0) for x in c.cached(b))
        pos = torch.arange(length - n, length, device=q.device)[:, None]
        j = torch.arange(length, device=q.device)[None]
        vis = j <= pos if causal else torch.ones(n, length, dtype=torch.bool, device=q.device)
        if gone is not None:
            vis = vis & ~gone[b][None]
            k, v = torch.where(gone[b][None, :, None], 0.0, k), torch.where(gone[b][None, :, None], 0.0, v)
        x = q[:, rows].double()
        p, _, _, _ = ref.weights(x @ k.transpose(1, 2) * scale, None, 0.0, vis)
        mag = abs(scale) * (x.abs() @ k.abs().transpose(1, 2))
        e = 2 * torch.where(vis, ref.score_error(None, mag), 0.0).amax(-1, keepdim=True)
        o[:, rows] = p @ v
        tol[:, rows] += (U + e) * (p @ v.abs() + o[:, rows].abs()) + U * o[:, rows].abs()
        tol[:, rows] += 2.0 ** -51 * torch.where(vis.any(0)[None, :, None], v.abs(), 0.0).amax((1, 2), keepdim=True)
    return o, tol
