"""GB300 (sm_103a) multi-head scaled dot-product attention forward.

A thin binding over the C ABI of libmha.so (include/mha.h): these functions
only marshal arguments -- every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and the stream.

    out = sdpa_forward(q, k, v, mask="causal")            # (B, h, T, 64) bf16
    out = sdpa_decode_forward(q, k_cache, v_cache, lens)   # (B, h, T_q <= 8, 64) bf16
    out = mha_forward(x_q, x_kv, w_q, w_k, w_v, w_o, h=8)  # (B, T, d_model) bf16

Every call runs on the current stream, or on the one passed as `stream`, which
then has to wait for the work that writes the call's inputs, as for any other
use of it (stream.wait_stream).  The tensors that a call makes itself are safe
on both: scratch belongs to the stream it is used on, results may be used (once
the current stream has waited) and dropped on the current one.
"""
from __future__ import annotations

import ctypes
import functools
import math

from . import _native
from ._native import (MHA_BF16, MHA_F32, MHA_MASK_CAUSAL, MHA_MASK_CAUSAL_KEY_PADDING,
                      MHA_MASK_KEY_PADDING, MHA_MASK_NONE, MHA_OK, lib)

__all__ = ["sdpa_forward", "sdpa_forward_lse", "sdpa_forward_host", "sdpa_forward_host_workspace_bytes",
           "sdpa_bf16_key_split", "sdpa_backward", "positional_encoding_add",
           "encoder_layer_forward", "ENCODER_PARAMS", "sdpa_decode_forward",
           "sdpa_scored_forward", "sdpa_scored_forward_lse", "sdpa_scored_backward",
           "sdpa_decode_shared_forward", "relative_bucket_starts", "mha_forward",
           "mha_forward_add_layernorm", "mha_workspace_bytes", "status_string", "MhaError", "MASKS", "lib"]

MASKS = {"none": MHA_MASK_NONE, "causal": MHA_MASK_CAUSAL, "key_padding": MHA_MASK_KEY_PADDING,
         "causal_key_padding": MHA_MASK_CAUSAL_KEY_PADDING}


class MhaError(RuntimeError):
    def __init__(self, code: int, what: str):
        detail = lib.mha_last_error().decode() if code == _native.MHA_ERR_CUDA else ""
        super().__init__("%s: %s (status %d)%s" % (what, status_string(code), code,
                                                   " -- " + detail if detail else ""))
        self.code = code


def status_string(code: int) -> str:
    return lib.mha_status_string(int(code)).decode()


def _mask_code(mask) -> int:
    if isinstance(mask, str):
        return MASKS[mask]
    return int(mask)


def _torch():
    import torch
    return torch


def _stream_handle(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _stream_on(stream, device):
    """_stream_handle for a device index, without building a Stream object (it
    costs a third of a small call's time on the host)."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(device)


def _result(stream, make, *args, **kwargs):
    """make(...), a tensor that the call's kernels write on `stream` and the
    caller gets.  The allocator orders a block's reuse by the stream it was
    allocated on, so a stream other than the current one allocates it (the
    block may still be in use by work queued on the current one otherwise), and
    its use on the current one is recorded, so that the caller may drop it there."""
    if stream is None:
        return make(*args, **kwargs)
    torch = _torch()
    current = torch.cuda.current_stream()
    if stream == current:
        return make(*args, **kwargs)
    with torch.cuda.stream(stream):
        t = make(*args, **kwargs)
    t.record_stream(current)
    return t


def _scratch(torch, workspace, need, device, stream):
    """(workspace, bytes): the caller's, or a new one of `need` bytes that
    belongs to `stream`: it is dropped as the call returns, with the kernels
    still to run, and only that stream's later work may have it then."""
    if workspace is None:
        if stream is None:
            return torch.empty(need or 1, dtype=torch.uint8, device=device), need
        with torch.cuda.stream(stream):
            return torch.empty(need or 1, dtype=torch.uint8, device=device), need
    _check_dev("workspace", workspace)
    return workspace, workspace.numel() * workspace.element_size()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_dev(name, t, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))


def sdpa_forward(q, k, v, out=None, *, scale=None, mask="none", key_lens=None, status=None,
                 stream=None):
    """softmax(scale * q k^T + mask) v for q (B,h,T_q,d_k), k (B,h,T_k,d_k),
    v (B,h,T_k,d_v); fp32 or bf16 CUDA tensors.  Returns out (B,h,T_q,d_v)."""
    torch = _torch()
    dtype = q.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("q must be float32 or bfloat16")
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_dev(n, t, dtype)
    B, h, T_q, d_k = q.shape
    T_k, d_v = k.shape[2], v.shape[3]
    if out is None:
        out = _result(stream, torch.empty, (B, h, T_q, d_v), dtype=dtype, device=q.device)
    _check_dev("out", out, dtype)
    if key_lens is not None:
        _check_dev("key_lens", key_lens, torch.int32)
    if status is not None:
        _check_dev("status", status, torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    rc = lib.sdpa_forward(MHA_F32 if dtype == torch.float32 else MHA_BF16, _ptr(q), _ptr(k),
                          _ptr(v), _ptr(out), B, h, T_q, T_k, d_k, d_v, float(scale),
                          _mask_code(mask), _ptr(key_lens), _ptr(status), _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_forward")
    return out


def sdpa_forward_lse(q, k, v, out=None, lse=None, *, scale=None, mask="none", key_lens=None,
                     status=None, stream=None):
    """sdpa_forward for bf16 tensors that also returns the per-row
    log-sum-exp of the visible scores, lse (B,h,T_q) fp32 (natural log; -inf
    for a row with no visible key).  Returns (out, lse)."""
    torch = _torch()
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_dev(n, t, torch.bfloat16)
    B, h, T_q, d_k = q.shape
    T_k, d_v = k.shape[2], v.shape[3]
    if out is None:
        out = _result(stream, torch.empty, (B, h, T_q, d_v), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = _result(stream, torch.empty, (B, h, T_q), dtype=torch.float32, device=q.device)
    _check_dev("out", out, torch.bfloat16)
    _check_dev("lse", lse, torch.float32)
    if key_lens is not None:
        _check_dev("key_lens", key_lens, torch.int32)
    if status is not None:
        _check_dev("status", status, torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    rc = lib.sdpa_forward_lse(MHA_BF16, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, h,
                              T_q, T_k, d_k, d_v, float(scale), _mask_code(mask), _ptr(key_lens),
                              _ptr(status), _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_forward_lse")
    return out, lse


def _check_host(name, t, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise ValueError("%s must be a CPU tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))


def sdpa_bf16_key_split(T_q, T_k, mask="none") -> int:
    """1 if the bf16 attention kernel splits a row's keys between its two
    softmax groups by alternate tiles for this shape, 0 if by key halves."""
    r = int(lib.sdpa_bf16_key_split(T_q, T_k, _mask_code(mask)))
    if r < 0:
        raise ValueError("invalid shape or mask")
    return r


def sdpa_forward_host_workspace_bytes(B, h, T_q, T_k, d_k=64, d_v=64, dtype=None) -> int:
    torch = _torch()
    dt = MHA_F32 if dtype == torch.float32 else MHA_BF16
    return int(lib.sdpa_forward_host_workspace_bytes(dt, B, h, T_q, T_k, d_k, d_v))


def sdpa_forward_host(q, k, v, out=None, workspace=None, *, scale=None, mask="none", key_lens=None,
                      status=None, stream=None):
    """sdpa_forward with q, k, v, out (and key_lens) in host memory (CPU
    tensors, page-locked for overlapped copies) and a device workspace; the
    library copies, computes and copies back in chunks that overlap.  The
    result is in `out` once `stream` has been synchronised.  Returns out."""
    torch = _torch()
    dtype = q.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("q must be float32 or bfloat16")
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_host(n, t, dtype)
    B, h, T_q, d_k = q.shape
    T_k, d_v = k.shape[2], v.shape[3]
    if out is None:
        out = torch.empty((B, h, T_q, d_v), dtype=dtype, pin_memory=torch.cuda.is_available())
    _check_host("out", out, dtype)
    if key_lens is not None:
        _check_host("key_lens", key_lens, torch.int32)
    if status is not None:
        _check_dev("status", status, torch.int32)
    dt = MHA_F32 if dtype == torch.float32 else MHA_BF16
    need = int(lib.sdpa_forward_host_workspace_bytes(dt, B, h, T_q, T_k, d_k, d_v))
    workspace, size = _scratch(torch, workspace, need, "cuda", stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    rc = lib.sdpa_forward_host(dt, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(workspace),
                               size, B, h, T_q, T_k, d_k,
                               d_v, float(scale), _mask_code(mask), _ptr(key_lens), _ptr(status),
                               _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_forward_host")
    return out


def sdpa_backward(q, k, v, o, dout, lse, dq=None, dk=None, dv=None, workspace=None, *,
                  scale=None, mask="none", key_lens=None, status=None, stream=None):
    """Gradients (dq, dk, dv) of sdpa_forward for bf16 tensors, from the
    forward's output o and log-sum-exp lse (sdpa_forward_lse) and the output
    gradient dout."""
    torch = _torch()
    bf = torch.bfloat16
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_dev(n, t, bf)
    _check_dev("lse", lse, torch.float32)
    B, h, T_q, d_k = q.shape
    T_k, d_v = k.shape[2], v.shape[3]
    dq = _result(stream, torch.empty_like, q) if dq is None else dq
    dk = _result(stream, torch.empty_like, k) if dk is None else dk
    dv = _result(stream, torch.empty_like, v) if dv is None else dv
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_dev(n, t, bf)
    need = int(lib.sdpa_backward_workspace_bytes(B, h, T_q, T_k, d_k, d_v))
    workspace, size = _scratch(torch, workspace, need, q.device, stream)
    if key_lens is not None:
        _check_dev("key_lens", key_lens, torch.int32)
    if status is not None:
        _check_dev("status", status, torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    rc = lib.sdpa_backward(MHA_BF16, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                           size, B, h, T_q, T_k, d_k,
                           d_v, float(scale), _mask_code(mask), _ptr(key_lens), _ptr(status),
                           _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_backward")
    return dq, dk, dv


def positional_encoding_add(x, out=None, *, pos0=0, stream=None):
    """x + PE(pos0 + t) for bf16 embedding rows x (B, T, d_model); out may be x."""
    torch = _torch()
    _check_dev("x", x, torch.bfloat16)
    B, T, D = x.shape
    out = _result(stream, torch.empty_like, x) if out is None else out
    _check_dev("out", out, torch.bfloat16)
    rc = lib.positional_encoding_add(_ptr(x), _ptr(out), B, T, D, int(pos0), _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "positional_encoding_add")
    return out


ENCODER_PARAMS = ("w_q", "w_k", "w_v", "w_o", "gamma1", "beta1", "w1", "b1", "w2", "b2", "gamma2",
                  "beta2")


def encoder_layer_forward(x, params, h, out=None, workspace=None, *, eps=1e-5, scale=None,
                          mask="none", key_lens=None, status=None, stream=None):
    """One post-LN encoder layer: y = LN1(x + MHA(x, x)), out = LN2(y + FFN(y)).
    params: dict of bf16 CUDA tensors named as ENCODER_PARAMS (W^Q..W^O
    (D, D), gamma/beta (D), w1 (D, F), b1 (F), w2 (F, D), b2 (D))."""
    torch = _torch()
    bf = torch.bfloat16
    _check_dev("x", x, bf)
    for n in ENCODER_PARAMS:
        _check_dev(n, params[n], bf)
    B, T, D = x.shape
    F = params["w1"].shape[1]
    out = _result(stream, torch.empty_like, x) if out is None else out
    _check_dev("out", out, bf)
    need = int(lib.encoder_layer_workspace_bytes(B, T, D, h, F))
    workspace, size = _scratch(torch, workspace, need, x.device, stream)
    if key_lens is not None:
        _check_dev("key_lens", key_lens, torch.int32)
    if status is not None:
        _check_dev("status", status, torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(D // h)
    rc = lib.encoder_layer_forward(_ptr(x), *[_ptr(params[n]) for n in ENCODER_PARAMS], float(eps),
                                   _ptr(out), _ptr(workspace),
                                   size, B, T, D, h, F,
                                   float(scale), _mask_code(mask), _ptr(key_lens), _ptr(status),
                                   _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "encoder_layer_forward")
    return out


def sdpa_decode_forward(q, k_cache, v_cache, cache_lens=None, out=None, *, scale=None,
                        stream=None):
    """Decoding step: each of the T_q (<= 8) query rows of q (B,h,T_q,64)
    attends to the first cache_lens[b] rows of k_cache / v_cache
    (B,h,T_k,64); bf16 CUDA tensors, cache_lens int32 on the device (None:
    all T_k).  Returns out (B,h,T_q,64)."""
    torch = _torch()
    for n, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_dev(n, t, torch.bfloat16)
    B, h, T_q, d_k = q.shape
    T_k, d_v = k_cache.shape[2], v_cache.shape[3]
    if out is None:
        out = _result(stream, torch.empty, (B, h, T_q, d_v), dtype=torch.bfloat16, device=q.device)
    _check_dev("out", out, torch.bfloat16)
    if cache_lens is not None:
        _check_dev("cache_lens", cache_lens, torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    rc = lib.sdpa_decode_forward(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), B, h, T_q,
                                 T_k, d_k, d_v, float(scale), _ptr(cache_lens),
                                 _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_decode_forward")
    return out


# ------------------------------------------------------------------ scored attention
def relative_bucket_starts(num_buckets, max_distance) -> tuple:
    """First distances of `num_buckets` relative position buckets (per
    direction): one bucket for each distance below num_buckets // 2, then
    logarithmically wider ones, bucket m + u (m = num_buckets // 2) starting at
    the first distance d with d / m >= (max_distance / m) ** (u / (num_buckets - m)).
    Computed in whole numbers, so no border depends on a rounding."""
    n, far = int(num_buckets), int(max_distance)
    near = n // 2
    if n < 2 or far < n:
        raise ValueError("num_buckets must be at least 2 and max_distance at least num_buckets")
    starts, d = list(range(near)), near
    for u in range(n - near):
        while d ** (n - near) < near ** (n - near - u) * far ** u:
            d += 1
        starts.append(max(d, starts[-1] + 1))
    return tuple(starts)


@functools.lru_cache(maxsize=64)
def _starts_array(starts):
    return (ctypes.c_int32 * len(starts))(*starts)


def _require(names, tensors, dtype, shape, device):
    """Each tensor that is not None is a contiguous CUDA tensor of that dtype,
    shape and device index.  (One call for all of a kind: on the host a small
    call's checks take as long as its launches.)"""
    for i, t in enumerate(tensors):
        if t is None:
            continue
        try:
            if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
                continue
        except AttributeError:
            pass
        _check_dev(names[i], t, dtype)
        if t.get_device() != device:
            raise ValueError("%s must be on cuda:%d, the current device" % (names[i], device))
        raise ValueError("%s must have the shape %s" % (names[i], tuple(shape)))


def _score_form(torch, h, B, T, device, cap, slopes, table, bucket_starts, prefix_lens, doc_ids, dtable=None):
    """(ScoreForm, the bucket starts' array it points into)."""
    f = _native.ScoreForm()
    keep = None
    if cap is not None:
        f.cap = cap
    if slopes is not None:
        _require(("slopes",), (slopes,), torch.float32, (h,), device)
        f.slopes = slopes.data_ptr()
    if (table is None) != (bucket_starts is None):
        raise ValueError("table and bucket_starts go together")
    if table is not None:
        keep = _starts_array(tuple(bucket_starts))
        n = len(keep)
        if n == 0 or not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] not in (n, 2 * n):
            raise ValueError("table must have one row per bucket, or two (bidirectional)")
        rows = table.shape[0]
        _require(("table", "dtable"), (table, dtable), torch.bfloat16, (rows, h), device)
        f.table = table.data_ptr()
        f.bucket_starts = ctypes.addressof(keep)
        f.num_buckets = n
        f.bidirectional = rows == 2 * n
    if prefix_lens is not None:
        _require(("prefix_lens",), (prefix_lens,), torch.int32, (B,), device)
        f.prefix_lens = prefix_lens.data_ptr()
    if doc_ids is not None:
        _require(("doc_ids",), (doc_ids,), torch.int32, (B, T), device)
        f.doc_ids = doc_ids.data_ptr()
    return f, keep


def _heads(torch, q, k, v, names, like):
    """Checked (B, h, h_kv, T_q, T_k, d, device index) of q (B, h, T_q, d), the
    tensors like it, and k, v (B, h_kv, T_k, d), bf16 on the current device.
    names: of k, v, q and the tensors like q."""
    device = torch.cuda.current_device()
    try:
        shape = q.shape
        B, h, T_q, d = shape
        _, h_kv, T_k, _ = k.shape
    except (AttributeError, ValueError):
        raise ValueError("%s and %s must be tensors of four dimensions" % (names[2], names[0])) from None
    if v is None:
        raise ValueError("%s must be a tensor" % names[1])
    _require(names[2:], (q, *like), torch.bfloat16, shape, device)
    _require(names, (k, v), torch.bfloat16, (B, h_kv, T_k, d), device)
    return B, h, h_kv, T_q, T_k, d, device


def _scratch_here(torch, workspace, need, device, stream):
    """_scratch on the current device, whose index is `device`."""
    workspace, size = _scratch(torch, workspace, need, device, stream)
    if workspace.get_device() != device:
        raise ValueError("workspace must be on cuda:%d, the current device" % device)
    return workspace, size


def _scored_call(torch, q, k, v, out, lse, out_lo, workspace, scale, cap, slopes, table, bucket_starts, mask,
                 key_lens, prefix_lens, doc_ids, status, stream, want_lse):
    B, h, h_kv, T_q, T_k, d, dev = _heads(torch, q, k, v, ("k", "v", "q", "out", "out_lo"), (out, out_lo))
    if out is None:
        out = _result(stream, torch.empty_like, q)
    if want_lse:
        if lse is None:
            lse = _result(stream, torch.empty, (B, h, T_q), dtype=torch.float32, device=dev)
        else:
            _require(("lse",), (lse,), torch.float32, (B, h, T_q), dev)
    if key_lens is not None:
        _require(("key_lens",), (key_lens,), torch.int32, (B,), dev)
    if status is not None:
        _check_dev("status", status, torch.int32)
    form, keep = _score_form(torch, h, B, T_k, dev, cap, slopes, table, bucket_starts, prefix_lens, doc_ids)
    pf = ctypes.addressof(form)
    size = 0
    if table is not None or doc_ids is not None or workspace is not None:
        workspace, size = _scratch_here(torch, workspace, lib.sdpa_scored_workspace_bytes(B, h, T_q, T_k, pf), dev, stream)
    rc = lib.sdpa_scored_forward(MHA_BF16, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse),
                                 _ptr(out_lo), _ptr(workspace), size, B, h, h_kv, T_q, T_k, d, d,
                                 1.0 / math.sqrt(d) if scale is None else scale, _mask_code(mask),
                                 _ptr(key_lens), pf, _ptr(status), _stream_on(stream, dev))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_scored_forward")
    return out, lse


def sdpa_scored_forward(q, k, v, out=None, workspace=None, *, scale=None, cap=None, slopes=None,
                        table=None, bucket_starts=None, mask="none", key_lens=None,
                        prefix_lens=None, doc_ids=None, status=None, stream=None):
    """Attention whose scores are scale q k^T, capped to cap tanh(./cap), plus a
    bias by distance (slopes: fp32 (h,), -slope |j - i|; or a learned table,
    bf16 (num_buckets [* 2], h), with the host sequence bucket_starts, see
    relative_bucket_starts), over the keys that mask, key_lens, prefix_lens
    (int32 (B,), with a causal mask) and doc_ids (int32 (B, T), not
    decreasing) leave.  q (B,h,T_q,64), k and v (B,h_kv,T_k,64) with h a
    multiple of h_kv; bf16.  Returns out (B,h,T_q,64)."""
    return _scored_call(_torch(), q, k, v, out, None, None, workspace, scale, cap, slopes, table, bucket_starts,
                        mask, key_lens, prefix_lens, doc_ids, status, stream, False)[0]


def sdpa_scored_forward_lse(q, k, v, out=None, lse=None, workspace=None, *, out_lo=None,
                            scale=None, cap=None, slopes=None, table=None, bucket_starts=None,
                            mask="none", key_lens=None, prefix_lens=None, doc_ids=None, status=None, stream=None):
    """sdpa_scored_forward that also returns the rows' log-sum-exp, lse
    (B,h,T_q) fp32, which sdpa_scored_backward takes.  out_lo: a tensor like
    out to receive what rounding took from it, for the backward's o_lo.
    Returns (out, lse)."""
    return _scored_call(_torch(), q, k, v, out, lse, out_lo, workspace, scale, cap, slopes, table, bucket_starts,
                        mask, key_lens, prefix_lens, doc_ids, status, stream, True)


def sdpa_scored_backward(q, k, v, o, dout, lse, dq=None, dk=None, dv=None, dtable=None,
                         workspace=None, *, o_lo=None, scale=None, cap=None, slopes=None,
                         table=None, bucket_starts=None, mask="none", key_lens=None,
                         prefix_lens=None, doc_ids=None, status=None, stream=None):
    """Gradients of sdpa_scored_forward from its output o (and the forward's
    out_lo, for exact row terms), log-sum-exp lse and the output gradient
    dout; every other argument as in the forward.  Returns
    (dq, dk, dv, dtable), dtable None without a table."""
    torch = _torch()
    B, h, h_kv, T_q, T_k, d, dev = _heads(torch, q, k, v, ("k", "v", "q", "o", "dout", "o_lo", "dq"),
                                          (o, dout, o_lo, dq))
    if o is None or dout is None or lse is None:
        raise ValueError("o, dout and lse are needed")
    _require(("lse",), (lse,), torch.float32, (B, h, T_q), dev)
    if dk is not None or dv is not None:
        _require(("dk", "dv"), (dk, dv), torch.bfloat16, k.shape, dev)
    if key_lens is not None:
        _require(("key_lens",), (key_lens,), torch.int32, (B,), dev)
    if status is not None:
        _check_dev("status", status, torch.int32)
    if table is None and dtable is not None:
        raise ValueError("dtable needs a table")
    form, keep = _score_form(torch, h, B, T_k, dev, cap, slopes, table, bucket_starts, prefix_lens, doc_ids, dtable)
    if dq is None:
        dq = _result(stream, torch.empty_like, q)
    if dk is None:
        dk = _result(stream, torch.empty_like, k)
    if dv is None:
        dv = _result(stream, torch.empty_like, v)
    if table is not None and dtable is None:
        dtable = _result(stream, torch.empty_like, table)
    pf = ctypes.addressof(form)
    workspace, size = _scratch_here(torch, workspace, lib.sdpa_scored_backward_workspace_bytes(B, h, h_kv, T_q, T_k, pf), dev,
                                    stream)
    rc = lib.sdpa_scored_backward(MHA_BF16, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(o_lo),
                                  dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                  _ptr(dtable), workspace.data_ptr(), size, B, h, h_kv, T_q, T_k, d, d,
                                  1.0 / math.sqrt(d) if scale is None else scale, _mask_code(mask),
                                  _ptr(key_lens), pf, _ptr(status), _stream_on(stream, dev))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_scored_backward")
    return dq, dk, dv, dtable


def sdpa_decode_shared_forward(q, k_prefix, v_prefix, k_cache, v_cache, cache_lens=None, out=None,
                               workspace=None, *, scale=None, cap=None, slopes=None, table=None,
                               bucket_starts=None, mask="none", status=None, stream=None):
    """Decoding step of a batch that shares a prefix: the T_q (<= 8) query rows
    of q (B,h,T_q,64) attend to every row of k_prefix / v_prefix (h_kv,T_p,64)
    and to the first cache_lens[b] rows of k_cache / v_cache (B,h_kv,T_k,64),
    whose last T_q they are; with a causal mask row t sees the cache up to its
    own row.  Scores as sdpa_scored_forward.  Returns out (B,h,T_q,64)."""
    torch = _torch()
    B, h, h_kv, T_q, T_k, d, dev = _heads(torch, q, k_cache, v_cache, ("k_cache", "v_cache", "q", "out"), (out,))
    try:
        _, T_p, _ = k_prefix.shape
    except (AttributeError, ValueError):
        raise ValueError("k_prefix must be a tensor of three dimensions") from None
    if v_prefix is None:
        raise ValueError("v_prefix must be a tensor")
    _require(("k_prefix", "v_prefix"), (k_prefix, v_prefix), torch.bfloat16, (h_kv, T_p, d), dev)
    if out is None:
        out = _result(stream, torch.empty_like, q)
    if cache_lens is not None:
        _require(("cache_lens",), (cache_lens,), torch.int32, (B,), dev)
    if status is not None:
        _check_dev("status", status, torch.int32)
    form, keep = _score_form(torch, h, B, T_k, dev, cap, slopes, table, bucket_starts, None, None)
    pf = ctypes.addressof(form)
    workspace, size = _scratch_here(torch, workspace, lib.sdpa_decode_shared_workspace_bytes(B, h, h_kv, T_q, T_p, T_k, pf), dev,
                                    stream)
    rc = lib.sdpa_decode_shared_forward(q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k_cache.data_ptr(),
                                        v_cache.data_ptr(), out.data_ptr(), workspace.data_ptr(), size, B, h, h_kv,
                                        T_q, T_p, T_k, d, d, 1.0 / math.sqrt(d) if scale is None else scale,
                                        _mask_code(mask), _ptr(cache_lens), pf, _ptr(status),
                                        _stream_on(stream, dev))
    if rc != MHA_OK:
        raise MhaError(rc, "sdpa_decode_shared_forward")
    return out


def mha_workspace_bytes(B, h, T_q, T_k, d_k=64, d_v=64) -> int:
    return int(lib.mha_workspace_bytes(B, h, T_q, T_k, d_k, d_v))


def _mha_call(x_q, x_kv, w_q, w_k, w_v, w_o, h, out, workspace, scale, mask, key_lens, status,
              stream, ln):
    torch = _torch()
    bf = torch.bfloat16
    for n, t in (("x_q", x_q), ("x_kv", x_kv), ("w_q", w_q), ("w_k", w_k), ("w_v", w_v),
                 ("w_o", w_o)):
        _check_dev(n, t, bf)
    B, T_q, D = x_q.shape
    T_k = x_kv.shape[1]
    d_k = w_q.shape[1] // h
    d_v = w_v.shape[1] // h
    if out is None:
        out = _result(stream, torch.empty, (B, T_q, D), dtype=bf, device=x_q.device)
    _check_dev("out", out, bf)
    need = mha_workspace_bytes(B, h, T_q, T_k, d_k, d_v)
    workspace, size = _scratch(torch, workspace, need, x_q.device, stream)
    if key_lens is not None:
        _check_dev("key_lens", key_lens, torch.int32)
    if status is not None:
        _check_dev("status", status, torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    ws = (_ptr(workspace), size)
    tail = (B, h, T_q, T_k, D, d_k, d_v, float(scale), _mask_code(mask), _ptr(key_lens),
            _ptr(status), _stream_handle(stream))
    if ln is None:
        rc = lib.mha_forward(MHA_BF16, _ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                             _ptr(w_o), _ptr(out), *ws, *tail)
        what = "mha_forward"
    else:
        gamma, beta, eps = ln
        _check_dev("gamma", gamma, bf)
        _check_dev("beta", beta, bf)
        if gamma.shape != (D,) or beta.shape != (D,):
            raise ValueError("gamma and beta must have d_model entries")
        rc = lib.mha_forward_add_layernorm(MHA_BF16, _ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(w_k),
                                           _ptr(w_v), _ptr(w_o), _ptr(gamma), _ptr(beta),
                                           float(eps), _ptr(out), *ws, *tail)
        what = "mha_forward_add_layernorm"
    if rc != MHA_OK:
        raise MhaError(rc, what)
    return out


def mha_forward(x_q, x_kv, w_q, w_k, w_v, w_o, h, out=None, workspace=None, *, scale=None,
                mask="none", key_lens=None, status=None, stream=None):
    """Concat_i(softmax(scale (x_q W_i^Q)(x_kv W_i^K)^T + mask)(x_kv W_i^V)) W^O
    for bf16 CUDA tensors x_q (B,T_q,D), x_kv (B,T_k,D) (may be x_q),
    W^Q/W^K/W^V (D, h*64), W^O (h*64, D).  Returns out (B,T_q,D)."""
    return _mha_call(x_q, x_kv, w_q, w_k, w_v, w_o, h, out, workspace, scale, mask, key_lens,
                     status, stream, None)


def mha_forward_add_layernorm(x_q, x_kv, w_q, w_k, w_v, w_o, gamma, beta, h, eps=1e-5,
                              out=None, workspace=None, *, scale=None, mask="none",
                              key_lens=None, status=None, stream=None):
    """LayerNorm(x_q + mha_forward(...)) with gain gamma and shift beta (bf16,
    d_model entries each): the attention sublayer with its residual
    connection and post-normalisation.  Returns out (B,T_q,D)."""
    return _mha_call(x_q, x_kv, w_q, w_k, w_v, w_o, h, out, workspace, scale, mask, key_lens,
                     status, stream, (gamma, beta, eps))
