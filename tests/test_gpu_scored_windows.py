"""Scores whose sums lie at opposite ends of what a row's reference serves (weights that sum to 2^-64 .. 2^64): key tiles
that go to different softmax groups, key ranges or launches, one with a reference far above its scores, one with a reference
far below, whose keys carry weights of a like size."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_reference as pr  # noqa: E402
import scored_reference as ref  # noqa: E402
from test_gpu_decode_shared import compare as compare_decode  # noqa: E402
from test_gpu_paged import compare as compare_paged  # noqa: E402
from test_gpu_scored import BF, gen, lib, run  # noqa: E402,F401

SCALE = math.log(2.0)  # a score of n is n in log2 units

# Scores of a tile's first and last 64 keys.  A round of 64 at -68 sums to 2^-62 against 0, which then is the row's reference;
# one at -130 sums to less than 2^-64 and moves it to -130, and one of -72.5 sums to 2^63.5 against that.  B's keys have
# 2^-4.5 of the weight of A's first 64.  C's have none beside them.
TILES = {"A": (-68.0, -200.0), "B": (-130.0, -72.5), "C": (-200.0, -200.0), "D": (-68.0, -68.0)}


def keys(tiles, g, lead, dtype=BF):
    """K and V (*lead, rows, 64): scores by the first feature, 2^-8 or less by the others; V of B's keys around 2."""
    s = torch.tensor([x for t in tiles for x in TILES[t] for _ in range(64)], device="cuda")
    far = torch.tensor([float(t == "B") for t in tiles for _ in range(128)], device="cuda")
    k = torch.randn(*lead, len(s), 64, generator=g, device="cuda") * 2.0 ** -12
    k[..., 0] = s
    v = torch.randn(*lead, len(s), 64, generator=g, device="cuda") * 0.25 + 2 * far[:, None]
    return k.to(dtype), v.to(dtype)


def rows(g, *shape):
    q = torch.randn(*shape, 64, generator=g, device="cuda") * 0.5
    q[..., 0] = 1.0
    return q.to(BF)


def forms(h):
    from transformer_scaled_dot_softmax_gb300 import relative_bucket_starts
    return {"plain": {}, "cap": {"cap": 1e6}, "slopes": {"slopes": torch.zeros(h, device="cuda")},
            "buckets": {"table": torch.zeros(8, h, dtype=BF, device="cuda"), "bucket_starts": relative_bucket_starts(8, 64)}}


@pytest.mark.parametrize("form", ["plain", "cap", "slopes", "buckets"])
@pytest.mark.parametrize("tiles", ["AB", "BA", "ACCB", "DB", "ABABAB", "BBA", "CAB" * 8, "AB" * 10])
def test_forward_and_gradients(lib, form, tiles):
    """Both forwards, the log-sum-exp and the gradients that follow from it."""
    g = gen(31)
    k, v = keys(tiles, g, (2, 2))
    q, go = rows(g, 2, 4, 130), torch.randn(2, 4, 130, 64, generator=g, device="cuda").to(BF)
    form = {"scale": SCALE, **forms(4)[form]}
    got = run(lib, q, k, v, go, form)
    want, fine = ref.attention(q, k, v, dout=go, **form), ref.attention(q, k, v, two_parts=True, **form)
    ref.check("o2", got["o2"], fine["o"], fine["o_tol"], 1)
    # dq elementwise alone: sum_j dS_ij = 0, so of the first feature's sum dS_ij k_j only what k_j differ by counts (4.5 of
    # 68), while each dS_ij is rounded times all of k_j; an average over the sums says nothing there.
    for n, m, roundings in (("o", "o", 2), ("lse", "lse", 1), ("dq", "dq", 0), ("dk", "dk", 2), ("dv", "dv", 2)):
        ref.check(n, got[n], want[m], want[m + "_tol"], roundings)


@pytest.mark.parametrize("form", ["plain", "cap", "slopes", "buckets"])
@pytest.mark.parametrize("prefix,cache", [("AB", ""), ("AB" * 20, "A"), ("AAAABBBB", "B"), ("A" * 9, "B" * 4), ("", "ABAB"),
                                          ("B" * 9, "A" * 9), ("C" * 30 + "AB", "BC")])
@pytest.mark.parametrize("shape", [(3, 4, 4, 1), (3, 4, 2, 1), (2, 2, 1, 5), (1, 4, 4, 2)])
def test_decoding_over_a_prefix(lib, form, prefix, cache, shape):
    """Groups of a key range, key ranges of the prefix and of the caches."""
    B, h, h_kv, T_q = shape
    g = gen(32)
    kp, vp = keys(prefix, g, (h_kv,))
    kc, vc = keys(cache, g, (B, h_kv))
    compare_decode(lib, (rows(g, B, h, T_q), kp, vp, kc, vc), None, {"scale": SCALE, **forms(h)[form]})


@pytest.mark.parametrize("tiles", ["AB", "BA", "ACCB", "AB" * 10, "A" * 9 + "B" * 9])
@pytest.mark.parametrize("new", [1, 3, 40, 130])
@pytest.mark.parametrize("capacity", [0, 40000])
def test_paged(lib, tiles, new, capacity):
    n = 128 * len(tiles)
    c = pr.Cache(2, 32, [n], [new], seed=33, capacity=capacity)
    c.rows = [keys(tiles, gen(33), (2,))]
    c.fill()
    compare_paged(lib, c, rows(gen(34), 4, new), False, scale=SCALE)
