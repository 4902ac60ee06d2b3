"""An int8 cache whose values are as small as its rows keep whole: as exact, relative to them, as any other."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import math  # noqa: E402

import paged_reference as pr  # noqa: E402
import scored_reference as ref  # noqa: E402
from test_gpu_paged import lib  # noqa: E402,F401

BF = torch.bfloat16


def rows(g, n, power, lift):
    """K: key 5 `lift` log2 units above the others, whose scores differ by less than 1; V: elements of 2^power / 2 to 2^power."""
    k = torch.randn(2, n, 64, generator=g, device="cuda") * 2.0 ** -5
    k[..., 0] = 0.0
    k[:, 5, 0] = lift
    v = (torch.rand(2, n, 64, generator=g, device="cuda") + 1) * 0.5
    v = torch.copysign(v, torch.randn(2, n, 64, generator=g, device="cuda") + 1)
    return k.to(BF), (v.to(BF).double() * 2.0 ** power).to(BF)


@pytest.mark.parametrize("power", [0, -60, -100, -110, -117, -119, 40, 45])
@pytest.mark.parametrize("lift", [0.0, 9.5, 13.0])
@pytest.mark.parametrize("new", [1, 4, 7, 40, 300])
@pytest.mark.parametrize("capacity", [0, 6000])
def test_values_of_every_size(lib, power, lift, new, capacity):
    """Against the definition at 2^0, of which this is a multiple: a row's bytes are the same and its exponent moves along
    (2^-119 holds rows whose exponent is -126, the least).  The output's own rounding is to multiples of 2^-133 below 2^-126."""
    n = 3000 if capacity else 900
    c = pr.Cache(2, 16, [n], [new], int8=True, seed=41, capacity=capacity)
    c.rows = [rows(c.g, n, power, lift)]
    c.fill()
    one = pr.Cache(2, 16, [n], [new], int8=True, seed=41, capacity=capacity)
    one.rows = [rows(one.g, n, 0, lift)]
    assert torch.equal(c.rows[0][0], one.rows[0][0])
    q = torch.randn(4, new, 64, generator=c.g, device="cuda") * 0.25
    q[..., 0] = 1.0
    q = q.to(BF)
    out = lib.sdpa_paged_forward(q, *c.args, c.row_starts, c.seq_lens, scale=math.log(2.0), max_new=new, **c.scales)
    want, tol = pr.attend(q, one, False, math.log(2.0))
    tol = tol + 2.0 ** (-134 - min(power, 0))
    ref.check("o", out.double() * 2.0 ** -power, want, tol, 0)
