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
