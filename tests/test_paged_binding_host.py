"""What the paged calls' binding makes of bounds and tensors at the edge of what it takes, with fakes of torch and the library."""
import pytest

from test_paged_host import Strided, fakes, nat, paged_calls  # noqa: F401
from test_stream_allocations_host import Lib


class Asked(Lib):
    """Remembers the arguments that attention was called with."""

    def __init__(self):
        super().__init__()
        self.most = []

    def sdpa_paged_workspace_bytes(self, cache, h, n, most):
        self.most.append(most)
        return 4096

    def sdpa_paged_forward(self, *a):
        self.most.append(a[11])
        return 0


def attend(m, **kw):
    return m.sdpa_paged_forward(Strided((4, 7, 64), "bfloat16"), Strided((9, 2, 16, 64), "bfloat16"),
                                Strided((9, 2, 16, 64), "bfloat16"), Strided((3, 5), "int32"), Strided((4,), "int32"),
                                Strided((3,), "int32"), **kw)


@pytest.mark.parametrize("most,taken", [(None, 7), (0, 0), (3, 3), (7, 7), (8, 7), (2 ** 31, 7), (2 ** 32 + 1, 7), (2 ** 63 - 1, 7)])
def test_a_bound_past_the_rows_is_their_number(fakes, monkeypatch, most, taken):
    """32 bits of a larger one would be another bound, 0 or 1 among them."""
    m, torch, _ = fakes
    lib = Asked()
    monkeypatch.setattr(m, "lib", lib)
    attend(m, max_new=most)
    assert lib.most == [taken, taken]


@pytest.mark.parametrize("most", [-1, -2 ** 32, -2 ** 32 + 1])
def test_a_bound_below_zero_is_refused(fakes, most):
    m, torch, lib = fakes
    with pytest.raises(ValueError):
        attend(m, max_new=most)
    assert lib.streams == []


PAGES = (Strided((9, 2, 16, 64), "bfloat16"), Strided((9, 2, 16, 64), "bfloat16"), Strided((3, 5), "int32"), Strided((3,), "int32"))


@pytest.mark.parametrize("kw", [{"k": 5}, {"k": Strided((3, 2), "bfloat16")}, {"k": Strided((3, 2, 80, 64), "float32")},
                                {"v": 5}, {"v": Strided((3, 2, 81, 64), "bfloat16")}, {"rows": -1},
                                {"rows": 7, "k": Strided((3, 2, 80, 64), "bfloat16")}])
def test_results_of_a_read_that_do_not_fit_are_refused(fakes, kw):
    m, torch, lib = fakes
    with pytest.raises(ValueError):
        m.paged_cache_read(*PAGES, **kw)
    assert lib.streams == [] and not torch.made


class Laid(Strided):
    """With strides of its own."""

    def __init__(self, shape, dtype, strides):
        super().__init__(shape, dtype)
        self.strides = strides

    def stride(self):
        return self.strides


# (shape, K's strides, V's): the stride of a dimension of size 1 means nothing, that of pages with one of them neither
ALIKE = [((1, 2, 16, 64), (2048, 1024, 64, 1), (4096, 1024, 64, 1)), ((9, 1, 16, 64), (1024, 1024, 64, 1), (1024, 77, 64, 1)),
         ((1, 1, 16, 64), (1024, 1024, 64, 1), (1, 1, 64, 1))]
UNLIKE = [((9, 2, 16, 64), (2048, 1024, 64, 1), (4096, 1024, 64, 1)), ((1, 2, 16, 64), (2048, 1024, 64, 1), (2048, 2048, 64, 1)),
          ((9, 1, 16, 64), (1024, 1024, 64, 1), (1024, 1024, 128, 1))]


@pytest.mark.parametrize("shape,ks,vs,taken", [(*x, True) for x in ALIKE] + [(*x, False) for x in UNLIKE])
def test_strides_that_count(fakes, shape, ks, vs, taken):
    m, torch, lib = fakes
    h_kv = shape[1]
    change = dict(k_pages=Laid(shape, "bfloat16", ks), v_pages=Laid(shape, "bfloat16", vs),
                  k=Strided((h_kv, 7, 64), "bfloat16"), v=Strided((h_kv, 7, 64), "bfloat16"))
    for name in ("append", "read", "attend"):
        if taken:
            paged_calls(m, **change)[name](None)
        else:
            with pytest.raises(ValueError):
                paged_calls(m, **change)[name](None)
    assert len(lib.streams) == (3 if taken else 0)
