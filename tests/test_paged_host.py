"""The paged K/V cache's calls on the host, without a GPU: what the C ABI and the binding refuse, workspace sizes, the order
and padding of mha_paged_cache, where the binding's allocations go, and the reference's 8-bit rows."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: every case below fails validation, or is empty


@pytest.fixture(scope="module")
def nat():
    import __graft_entry__
    __graft_entry__.build()
    from transformer_scaled_dot_softmax_gb300 import _native
    return _native


def cache(nat, **kw):
    f = dict(dtype=nat.MHA_BF16, k_pages=FAKE, v_pages=FAKE, page_stride=4 * 16 * 64, k_scales=None, v_scales=None,
             page_table=FAKE, row_starts=FAKE, seq_lens=FAKE, B=2, h_kv=4, page_rows=16, num_pages=10, max_pages=80)
    f.update(kw)
    return nat.PagedCache(**f)


def append(nat, c, k=FAKE, kh=64 * 5, kt=64, v=FAKE, vh=64 * 5, vt=64, N=5, d=64):
    return nat.lib.paged_cache_append(ctypes.addressof(c) if c else None, k, kh, kt, v, vh, vt, N, d, None)


def read(nat, c, k=FAKE, v=FAKE, T=20, d=64):
    return nat.lib.paged_cache_read(ctypes.addressof(c) if c else None, k, v, T, d, None)


def attend(nat, c, q=FAKE, qh=64 * 5, qt=64, o=FAKE, oh=64 * 5, ot=64, ws=FAKE, size=1 << 40, h=8, N=5, most=5, d=64, scale=0.125,
           mask=1):
    return nat.lib.sdpa_paged_forward(ctypes.addressof(c) if c else None, q, qh, qt, o, oh, ot, ws, size, h, N, most, d, scale,
                                      mask, None, None)


CALLS = [append, read, attend]


@pytest.mark.parametrize("call", CALLS)
def test_caches_that_are_refused(nat, call):
    bad = nat.MHA_ERR_INVALID_ARG
    assert call(nat, None) == bad
    for field in ("k_pages", "v_pages", "page_table", "seq_lens"):
        assert call(nat, cache(nat, **{field: None})) == bad, field
    for field in ("B", "h_kv", "num_pages", "max_pages", "page_rows"):
        assert call(nat, cache(nat, **{field: -1})) == bad, field
    assert call(nat, cache(nat, dtype=7)) == bad
    assert call(nat, cache(nat, page_rows=0)) == bad
    assert call(nat, cache(nat, dtype=nat.MHA_F32)) == nat.MHA_ERR_UNSUPPORTED
    assert call(nat, cache(nat), d=32) == nat.MHA_ERR_UNSUPPORTED
    assert call(nat, cache(nat), d=0) == bad
    for rows in (8, 24, 100, 65536 + 16):
        assert call(nat, cache(nat, page_rows=rows, page_stride=1 << 30)) == nat.MHA_ERR_UNSUPPORTED, rows
    # pages that overlap, or that TMA could not address
    assert call(nat, cache(nat, page_stride=4 * 16 * 64 - 16)) == bad
    assert call(nat, cache(nat, page_stride=4 * 16 * 64 + 8)) == bad
    assert call(nat, cache(nat, page_stride=1 << 38)) == nat.MHA_ERR_UNSUPPORTED
    assert call(nat, cache(nat, max_pages=1 << 26)) == nat.MHA_ERR_UNSUPPORTED
    assert call(nat, cache(nat, k_pages=FAKE + 8)) == nat.MHA_ERR_MISALIGNED
    assert call(nat, cache(nat, v_pages=FAKE + 2)) == nat.MHA_ERR_MISALIGNED
    int8 = dict(dtype=nat.MHA_INT8, k_scales=FAKE, v_scales=FAKE)
    for field in ("k_scales", "v_scales"):
        assert call(nat, cache(nat, **{**int8, field: None})) == bad
        assert call(nat, cache(nat, **{**int8, field: FAKE + 1})) == nat.MHA_ERR_MISALIGNED


def test_rows_that_are_refused(nat):
    bad, c = nat.MHA_ERR_INVALID_ARG, cache(nat)
    assert append(nat, cache(nat, row_starts=None)) == bad
    assert attend(nat, cache(nat, row_starts=None)) == bad
    assert append(nat, c, N=-1) == bad and attend(nat, c, N=-1) == bad and read(nat, c, T=-1) == bad
    for p in ("k", "v"):
        assert append(nat, c, **{p: None}) == bad
        assert append(nat, c, **{p: FAKE + 8}) == nat.MHA_ERR_MISALIGNED
        assert read(nat, c, **{p: None}) == bad
        assert read(nat, c, **{p: FAKE + 8}) == nat.MHA_ERR_MISALIGNED
        for s in ("h", "t"):  # heads or rows on top of one another, and off their 16 bytes
            assert append(nat, c, **{p + s: 0}) == bad
            assert append(nat, c, **{p + s: -64}) == bad
            assert append(nat, c, **{p + s: 68}) == nat.MHA_ERR_MISALIGNED
            assert append(nat, c, **{p + s: 1 << 38}) == nat.MHA_ERR_UNSUPPORTED
    for p in ("q", "o"):
        assert attend(nat, c, **{p: None}) == bad
        assert attend(nat, c, **{p: FAKE + 8}) == nat.MHA_ERR_MISALIGNED
        for s in ("h", "t"):
            assert attend(nat, c, **{p + s: 0}) == bad
            assert attend(nat, c, **{p + s: 72 + 4}) == nat.MHA_ERR_MISALIGNED


def test_attention_that_is_refused(nat):
    bad, c = nat.MHA_ERR_INVALID_ARG, cache(nat)
    for h in (-1, 6):  # not a multiple of the K/V heads
        assert attend(nat, c, h=h) == bad
    assert attend(nat, cache(nat, h_kv=0)) == bad
    assert attend(nat, cache(nat, h_kv=1, page_stride=1 << 12), h=129) == nat.MHA_ERR_UNSUPPORTED
    assert attend(nat, c, most=-1) == bad
    assert attend(nat, c, mask=4) == bad and attend(nat, c, mask=-1) == bad
    for scale in (float("nan"), float("inf"), 3e38):
        assert attend(nat, c, scale=scale) == bad
    assert attend(nat, c, N=1 << 28, qh=64 << 28, oh=64 << 28) == nat.MHA_ERR_UNSUPPORTED
    # work that 32 bits do not number
    assert attend(nat, cache(nat, B=60000, max_pages=1 << 20)) == nat.MHA_ERR_UNSUPPORTED
    need = nat.lib.sdpa_paged_workspace_bytes(ctypes.addressof(c), 8, 5, 5)
    assert attend(nat, c, ws=None) == nat.MHA_ERR_WORKSPACE
    assert attend(nat, c, size=need - 1) == nat.MHA_ERR_WORKSPACE
    assert attend(nat, c, ws=FAKE + 16) == nat.MHA_ERR_MISALIGNED


def test_empty_calls_do_nothing(nat):
    for call in (append, attend):
        assert call(nat, cache(nat), N=0) == nat.MHA_OK
        assert call(nat, cache(nat, B=0, seq_lens=None, row_starts=None, page_table=None)) == nat.MHA_OK
    assert read(nat, cache(nat), T=0) == nat.MHA_OK
    assert read(nat, cache(nat, B=0, seq_lens=None)) == nat.MHA_OK
    assert append(nat, cache(nat, max_pages=0, page_table=None)) == nat.MHA_OK  # nowhere to put a row
    assert append(nat, cache(nat, num_pages=0, k_pages=None, v_pages=None)) == nat.MHA_OK
    assert attend(nat, cache(nat), most=0) == nat.MHA_OK
    assert attend(nat, cache(nat), h=0) == nat.MHA_OK


def test_workspace_sizes(nat):
    def need(c, h=8, N=5, most=5):
        return nat.lib.sdpa_paged_workspace_bytes(ctypes.addressof(c), h, N, most)

    assert nat.lib.sdpa_paged_workspace_bytes(None, 8, 5, 5) == 0
    for kw in (dict(h=7), dict(N=-1), dict(most=-1), dict(N=0), dict(most=0), dict(h=0)):
        assert need(cache(nat), **kw) == 0
    assert need(cache(nat, page_rows=8)) == 0
    # sizes alone count
    assert need(cache(nat, k_pages=None, v_pages=None, page_table=None, seq_lens=None, row_starts=None)) == need(cache(nat))
    # none where every item is one CTA's: few query rows of short sequences
    assert need(cache(nat, max_pages=64)) == 0 < need(cache(nat, max_pages=65))
    assert need(cache(nat, max_pages=64), N=17, most=17) > 0
    # it grows with the rows that may have to be stacked, and an int8 chunk's cache has room as bf16
    small, chunk = need(cache(nat), N=600, most=1), need(cache(nat, page_rows=64, page_stride=4 * 64 * 64), N=600, most=600)
    assert 0 < small < chunk
    wide = need(cache(nat, dtype=nat.MHA_INT8, page_rows=64, page_stride=4 * 64 * 64), N=600, most=600)
    assert wide >= chunk + 2 * 2 * 4 * (80 * 64) * 64 * 2
    # ... up to 4 GiB of it
    huge = cache(nat, dtype=nat.MHA_INT8, B=64, page_rows=64, page_stride=4 * 64 * 64, max_pages=1 << 14)
    assert need(huge, N=60000, most=600) < 1 << 30


def test_the_binding_packs_the_declared_struct(nat):
    """Offsets of the packed bytes are those of the ctypes structure, whose fields are those of the header, in order."""
    text = open(os.path.join(ROOT, "include", "mha.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} mha_paged_cache;", text).group(1)
    names = re.findall(r"[*\s](\w+)(?=[,;])", body)
    assert names == [n for n, _ in nat.PagedCache._fields_]
    values = list(range(3, 3 + len(names)))
    c = nat.PagedCache.from_buffer_copy(nat.pack_paged_cache(*values).ljust(ctypes.sizeof(nat.PagedCache), b"\0"))
    assert [getattr(c, n) for n in names] == values
    assert ctypes.sizeof(nat.PagedCache) - len(nat.pack_paged_cache(*values)) < 8


# ----------------------------------------------------------------------------------------- the binding, with fakes of torch
from test_stream_allocations_host import Lib, Stream, Tensor, Torch  # noqa: E402


class Strided(Tensor):
    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)


@pytest.fixture
def fakes(monkeypatch, nat):
    import transformer_scaled_dot_softmax_gb300 as m
    torch, lib = Torch(), Lib()
    torch.int8 = "int8"
    make = torch.empty

    def empty(*a, **kw):
        t = make(*a, **kw)
        s = Strided(t.shape, t.dtype, t.owner)
        torch.made[-1] = s
        return s

    torch.empty = empty
    torch.empty_like = lambda t: empty(t.shape, dtype=t.dtype)
    monkeypatch.setattr(m, "_torch", lambda: torch)
    monkeypatch.setattr(m, "lib", lib)
    return m, torch, lib


def paged_calls(m, **change):
    t = dict(k=Strided((2, 7, 64), "bfloat16"), v=Strided((2, 7, 64), "bfloat16"), q=Strided((4, 7, 64), "bfloat16"),
             k_pages=Strided((9, 2, 16, 64), "bfloat16"), v_pages=Strided((9, 2, 16, 64), "bfloat16"),
             page_table=Strided((3, 5), "int32"), row_starts=Strided((4,), "int32"), seq_lens=Strided((3,), "int32"),
             k_scales=None, v_scales=None)
    t.update(change)
    pages, scales = (t["k_pages"], t["v_pages"], t["page_table"]), {"k_scales": t["k_scales"], "v_scales": t["v_scales"]}
    return {"append": lambda s: m.paged_cache_append(t["k"], t["v"], *pages, t["row_starts"], t["seq_lens"], stream=s, **scales),
            "read": lambda s: m.paged_cache_read(*pages, t["seq_lens"], stream=s, **scales),
            "attend": lambda s: m.sdpa_paged_forward(t["q"], *pages, t["row_starts"], t["seq_lens"], stream=s, **scales)}


@pytest.mark.parametrize("name,results,scratch", [("append", 0, 0), ("read", 2, 0), ("attend", 1, 1)])
def test_allocations_follow_the_named_stream(fakes, name, results, scratch):
    m, torch, lib = fakes
    side = Stream(9)
    made = paged_calls(m)[name](side)
    made = made if isinstance(made, tuple) else (made,)
    assert lib.streams == [9]
    assert len(torch.made) == results + scratch and all(t.owner == side for t in torch.made)
    for t in torch.made:
        assert t.uses == ([torch.current] if any(t is r for r in made) else [])
    paged_calls(m)[name](None)
    paged_calls(m)[name](torch.current)
    assert lib.streams == [9, 7, 7]
    assert all(t.owner == torch.current and not t.uses for t in torch.made[results + scratch:])


OTHER = [("page_table", (4, 5), "int32"), ("page_table", (3, 5), "int64"), ("page_table", (15,), "int32"),
         ("row_starts", (3,), "int32"), ("row_starts", (4,), "int64"), ("seq_lens", (4,), "int32"), ("seq_lens", (3, 1), "int32"),
         ("seq_lens", (3,), "float32"), ("v_pages", (9, 2, 16, 32), "bfloat16"), ("v_pages", (9, 2, 16, 64), "int8"),
         ("k_pages", (9, 2, 1024), "bfloat16"), ("k_pages", (9, 2, 16, 64), "float32"), ("k", (3, 7, 64), "bfloat16"),
         ("k", (2, 7, 64), "float32"), ("v", (2, 6, 64), "bfloat16"), ("q", (4, 7, 32), "bfloat16"), ("q", (4, 448), "bfloat16")]


@pytest.mark.parametrize("field,shape,dtype", OTHER)
def test_the_binding_refuses(fakes, field, shape, dtype):
    m, torch, lib = fakes
    uses = {"k": ["append"], "v": ["append"], "q": ["attend"], "row_starts": ["append", "attend"]}.get(
        field, ["append", "read", "attend"])
    for name in uses:
        with pytest.raises(ValueError):
            paged_calls(m, **{field: Strided(shape, dtype)})[name](None)
    for name in uses:
        for nothing in (None, 5):
            with pytest.raises(ValueError):
                paged_calls(m, **{field: nothing})[name](None)
    assert lib.streams == []


def test_the_binding_refuses_scales_that_do_not_fit(fakes):
    m, torch, lib = fakes
    s = Strided((9, 2, 16), "uint8")
    pages = dict(k_pages=Strided((9, 2, 16, 64), "int8"), v_pages=Strided((9, 2, 16, 64), "int8"))
    for change in (dict(k_scales=s), dict(k_scales=s, v_scales=s), dict(**pages), dict(k_scales=s, **pages),
                   dict(k_scales=s, v_scales=Strided((9, 2, 32), "uint8"), **pages),
                   dict(k_scales=s, v_scales=Strided((9, 2, 16), "int8"), **pages)):
        for name in ("append", "read", "attend"):
            with pytest.raises(ValueError):
                paged_calls(m, **change)[name](None)
    assert lib.streams == []
    for name in ("append", "read", "attend"):
        paged_calls(m, k_scales=s, v_scales=s, **pages)[name](None)


# ------------------------------------------------------------------------------------------------------- 8-bit rows
def test_the_reference_rows_are_the_definition():
    """stored() against whole-number arithmetic on bf16's own bits: the exponent from the largest element's bits, ties by
    comparing remainders."""
    torch = pytest.importorskip("torch")
    import paged_reference as pr
    g = torch.Generator().manual_seed(1)
    x = torch.randn(400, 64, generator=g) * torch.exp2(torch.randint(-133, 120, (400, 1), generator=g).float())
    x[::7] = torch.round(x[::7] / x[::7].abs().amax(1, keepdim=True) * 254) / 2  # halves
    x = x.to(torch.bfloat16)
    n, s = pr.stored(x)
    for row, kept, e in zip(x.tolist(), n.tolist(), s.tolist()):
        from fractions import Fraction
        exact = [Fraction(v) for v in row]
        step = Fraction(2) ** (e - 127)
        top = max(abs(v) for v in exact)
        assert top <= 127 * step and (e == 1 or top > 127 * step / 2)
        for v, k in zip(exact, kept):
            q = v / step
            down = q.numerator // q.denominator
            rest = q - down
            up = rest > Fraction(1, 2) or (rest == Fraction(1, 2) and down % 2)
            assert k == (down + 1 if up else down)
    assert torch.equal(pr.values(n, s).to(torch.bfloat16).double(), pr.values(n, s))
