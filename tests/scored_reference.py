"""Scored attention, its gradients and shared-prefix decoding from the definition, in fp64 torch, with elementwise
bounds on what the library's roundings may change.

Bounds.  u = 2^-8 is the relative rounding of one bf16 rounding (half a step), w the exact weights.
  weights  A weight enters P V after a score error e_s, |e_s| <= SCORE (below), and rounded to bf16 (r = u), or with lse
           as two bf16 parts (r = u^2); numerator and normaliser use the same weights, so o moves by at most
           (r + e) (sum w |v| + |o|), e = 2 e_s, and is rounded once: u |o|.
  lse      ln of the sum of the weights: e absolute, plus fp32.
  P        recomputed as exp(s - lse): relative 2 e (score and lse), and rounded for dV: u.
  D        sum dO o of the library's o + o_lo: the weights' errors d_j move it by sum d_j w_j (dP_j - D), at most
           (u^2 + e) sum |dS|, the pair's own rounding by u^2 sum |dO| |o|; without o_lo by u sum |dO| |o|.
  dS       relative 2 e, and P |dD|; rounded: u.  dP and D are fp32 sums of 64 products: 2^-16 of sum |dO| |v|.
  dq, dk, dv, dtable: the sums of those, rounded once more (u).
A second check on the relative 2-norm takes each rounding at its mean square, u / sqrt(3), in quadrature (check's
`roundings`).  That is an average: it holds where the tensor comes of many rows, and the check is left out below 64.  Nor
for dtable: it holds sums of dS over buckets, and sum_j dS_ij = 0, so a bucket with most of a row's weight sums to little,
while D's error enters it with sum_j P_ij = 1; there the elementwise bound alone stands.
"""
import math

import torch

U = 2.0 ** -8


def score_error(cap, s_abs):
    """Bound of the error of one score: fp32 products and sums of 64 terms and the bias (2^-18 of the magnitudes),
    the capping polynomials (2.2e-5 of a score below cap / 2, 2.2e-6 cap above), 2^x (2^-21 relative)."""
    return 2.0 ** -18 * s_abs + ((2.2e-5 * s_abs).clamp(max=1.1e-5 * cap) + 3e-6 * cap if cap else 0.0) + 2.0 ** -20


def bucket_of(d, starts, both):
    away = d.abs() if both else (-d).clamp(min=0)
    b = torch.zeros_like(d)
    for u, s in enumerate(starts):
        b = torch.where(away >= s, torch.full_like(b, u), b)
    return b + (len(starts) * (d > 0) if both else 0)


def bias_of(d, h, slopes, table, starts):
    """(h, *d.shape) fp64."""
    if slopes is not None:
        return -slopes.double().reshape(h, *[1] * d.dim()) * d.abs()
    if table is not None:
        return table.double().t()[:, bucket_of(d, starts, table.shape[0] == 2 * len(starts))]
    return torch.zeros((h,) + tuple(1 for _ in d.shape), dtype=torch.float64, device=d.device)


def visible(B, T_q, T_k, dev, mask, key_lens=None, prefix_lens=None, doc_ids=None):
    i, j = torch.arange(T_q, device=dev)[:, None], torch.arange(T_k, device=dev)[None]
    vis = torch.ones(B, T_q, T_k, dtype=torch.bool, device=dev)
    if "causal" in mask:
        see = (j <= i)[None].expand(B, T_q, T_k)
        if prefix_lens is not None:
            see = see | (j[None] < prefix_lens.long()[:, None, None])
        vis = vis & see
    if "key_padding" in mask:
        vis = vis & (j[None] < key_lens.long()[:, None, None])
    if doc_ids is not None:
        vis = vis & (doc_ids[:, :, None] == doc_ids[:, None, :])
    return vis


def weights(z, cap, bias, vis):
    """(P, t, lse, scores) of products z (already scaled)."""
    t = torch.tanh(z / cap) if cap else None
    s = (cap * t if cap else z) + bias
    s = torch.where(vis, s, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(vis, torch.exp(s - torch.where(lse.isfinite(), lse, 0.0)[..., None]), 0.0)
    return p, t, lse, s


def attention(q, k, v, *, scale, cap=None, slopes=None, table=None, bucket_starts=None, mask="none", key_lens=None,
              prefix_lens=None, doc_ids=None, dout=None, o_lo=True, two_parts=False):
    """dict of exact values and, under the same names with "_tol", elementwise bounds."""
    B, h, T_q, d = q.shape
    h_kv, T_k = k.shape[1], k.shape[2]
    g = h // h_kv
    vis = visible(B, T_q, T_k, q.device, mask, key_lens, prefix_lens, doc_ids)[:, None]
    live = vis.any(2)  # (B, 1, T_k): keys that count at all
    q, k, v = q.double(), k.double(), v.double()
    k, v = torch.where(live[..., None], k, 0.0), torch.where(live[..., None], v, 0.0)
    ke, ve = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    dist = torch.arange(T_k, device=q.device)[None] - torch.arange(T_q, device=q.device)[:, None]
    z = q @ ke.transpose(2, 3) * scale
    bias = bias_of(dist, h, slopes, table, bucket_starts)
    p, t, lse, s = weights(z, cap, bias, vis)
    mag = abs(scale) * (q.abs() @ ke.abs().transpose(2, 3)) + bias.abs()
    e = 2 * torch.where(vis, score_error(cap, mag), 0.0).amax(-1, keepdim=True)
    # weights that vanish beside their row's largest are flushed or underflow: 2^-120 of it at most
    r = {"o": p @ ve, "lse": lse}
    r["o_tol"] = ((U * U if two_parts else U) + e) * (p @ ve.abs() + r["o"].abs()) + U * r["o"].abs() + 1e-30
    r["lse_tol"] = e[..., 0] + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)
    if dout is None:
        return r
    go = dout.double()
    dp = go @ ve.transpose(2, 3)
    D = (go * r["o"]).sum(-1, keepdim=True)
    ds = p * (dp - D)
    D_tol = 1.02 * (U * U + e) * ds.abs().sum(-1, keepdim=True) + (2.0 ** -15 if o_lo else U) * (go.abs() * r["o"].abs()).sum(-1, keepdim=True)
    dp_tol = 2.0 ** -16 * (go.abs() @ ve.abs().transpose(2, 3))
    ds_tol = 2 * e * 1.05 * ds.abs() + 1.05 * p * (D_tol + dp_tol)
    f = 1.0 if t is None else 1 - t * t
    dz = ds * f
    # 1 - t^2 of the polynomial's t: 6e-6 absolute
    dz_tol = (ds_tol * f + 6e-6 * ds.abs() + U * (dz.abs() + ds_tol)) if t is not None else ds_tol + U * (ds.abs() + ds_tol)

    def shared(x):
        return x.reshape(B, h_kv, g, T_k, d).sum(2)

    r["dq"] = scale * (dz @ ke)
    r["dq_tol"] = abs(scale) * (dz_tol @ ke.abs())
    r["dk"] = shared(scale * (dz.transpose(2, 3) @ q))
    r["dk_tol"] = shared(abs(scale) * (dz_tol.transpose(2, 3) @ q.abs()))
    r["dv"] = shared(p.transpose(2, 3) @ go)
    p_tol = (U + 2 * e) * 1.05 * p
    r["dv_tol"] = shared(p_tol.transpose(2, 3) @ go.abs())
    if table is not None:
        n = table.shape[0]
        b = bucket_of(dist, bucket_starts, n == 2 * len(bucket_starts)).reshape(-1)

        def by_bucket(x):
            return torch.zeros(n, h, dtype=torch.float64, device=q.device).index_add_(0, b, x.sum(0).reshape(h, -1).t())

        r["dtable"], r["dtable_tol"] = by_bucket(ds), by_bucket(ds_tol + 2.0 ** -20 * ds.abs())
    for n in ("dq", "dk", "dv", "dtable"):
        if n in r:
            r[n + "_tol"] = r[n + "_tol"] * (1 + U) + U * r[n].abs() + 1e-30
    return r


def decode(q, k_prefix, v_prefix, k_cache, v_cache, cache_lens, *, scale, cap=None, slopes=None, table=None,
           bucket_starts=None, mask="none"):
    B, h, T_q, _ = q.shape
    h_kv, T_k = k_cache.shape[1], k_cache.shape[2]
    P, g, dev = k_prefix.shape[1], h // h_kv, q.device
    o, tol = torch.zeros(q.shape, dtype=torch.float64, device=dev), torch.zeros(q.shape, dtype=torch.float64, device=dev)
    for b in range(B):
        n = T_k if cache_lens is None else min(max(int(cache_lens[b]), 0), T_k)
        ke = torch.cat((k_prefix, k_cache[b, :, :n]), 1).double().repeat_interleave(g, 0)
        ve = torch.cat((v_prefix, v_cache[b, :, :n]), 1).double().repeat_interleave(g, 0)
        t = torch.arange(T_q, device=dev)
        pos, j = (P + n - T_q + t)[:, None], torch.arange(P + n, device=dev)[None]
        vis = (j <= pos) | (j < P) if "causal" in mask else torch.ones(T_q, P + n, dtype=torch.bool, device=dev)
        bias = bias_of(j - pos, h, slopes, table, bucket_starts)
        x = q[b].double()
        p, _, _, _ = weights(x @ ke.transpose(1, 2) * scale, cap, bias, vis)
        mag = abs(scale) * (x.abs() @ ke.abs().transpose(1, 2)) + bias.abs()
        e = 2 * torch.where(vis, score_error(cap, mag), 0.0).amax(-1, keepdim=True) if P + n else torch.zeros(h, T_q, 1, device=dev)
        o[b] = p @ ve
        tol[b] = (U + e) * (p @ ve.abs() + o[b].abs()) + U * o[b].abs() + 1e-30
    return o, tol


def check(name, got, ref, tol, roundings, rows=64):
    got = got.double()
    assert bool(torch.isfinite(got).all()) or not bool(torch.isfinite(ref).all()), name + ": not finite"
    fin = torch.isfinite(ref)
    assert torch.equal(got[~fin], ref[~fin]), name + ": infinities differ"
    off = (got - ref)[fin].abs()
    worst = (off / tol[fin]).max().item() if off.numel() else 0.0
    assert worst <= 1, "%s: %.3g of the bound (largest error %.3g, |ref| up to %.3g)" % (
        name, worst, off.max().item(), ref[fin].abs().max().item())
    norm = ref[fin].norm().item()
    if roundings and rows >= 64 and norm > 1e-3 * math.sqrt(max(off.numel(), 1)):
        rel = off.norm().item() / norm
        assert rel <= U * math.sqrt(roundings / 3.0), "%s: relative error %.3g" % (name, rel)
