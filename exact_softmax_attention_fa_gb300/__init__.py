"""GB300 (sm_103a) exact softmax attention: Python binding of the C ABI.

The functions here only check and marshal arguments (torch tensors -> device
pointers, sizes, the current CUDA stream) and call libfa_gb300.so; every step
of the computation runs in the library's CUDA kernels. PyTorch supplies device
memory and streams.

    o, lse = forward(q, k, v, causal=True)            # q, k, v: bf16 [B, H, N, d] on CUDA
    dq, dk, dv = backward(q, k, v, o, lse, do, causal=True)
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import threading

from ._lib import load, check, FAError, header_functions, STATUS_NAMES  # noqa: F401

__all__ = ["fa_fwd", "fa_bwd", "fa_fwd_gqa", "fa_bwd_gqa", "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_size", "fa_bwd_deterministic", "fa_bwd_gqa_deterministic", "fa_bwd_workspace_size", "fa_bwd_gqa_workspace_size", "fa_bwd_preprocess", "fa_bwd_preprocess_stats", "fa_bwd_main", "fa_bwd_postprocess", "fa_bwd_dkdv", "fa_bwd_dq", "fa_bwd_noalloc", "fa_fwd_bwd_host", "fa_fwd_bwd_host_device_bytes", "fa_fwd_host", "fa_fwd_host_device_bytes", "fa_get_device_status", "fa_get_device_status_detail", "fa_set_wait_limit_ns",
           "fa_debug_timeout_probe", "fa_debug_skip_arrival", "fa_norm_rope_fwd", "fa_norm_rope_bwd",
           "fa_norm_rope_bwd_workspace_size", "fa_kv8_append", "fa_kv8_advance", "fa_kv8_gather",
           "fa_fwd_kv8", "fa_fwd_kv8_filled", "fa_fwd_kv8_workspace_size", "KV8Cache", "rope_tables", "norm_rope", "norm_rope_backward", "forward", "backward", "FAError", "flops"]

_SUPPORTED_D = (64, 128, 256)


def _stream_handle(stream):
    import torch
    if stream is None:  # the handle alone: building torch's stream object takes longer than a launch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dims(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(int(x) for x in q.shape)


def _check_bf16(name, t, shape):
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _check_lse(t, shape):
    import torch
    if t.dtype != torch.float32 or tuple(t.shape) != shape[:3] or not t.is_cuda or not t.is_contiguous():
        raise ValueError("lse must be a contiguous float32 CUDA tensor of shape [B, H, N]")


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def fa_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """fa_fwd of the C ABI on torch tensors (outputs o, lse written in place)."""
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check_bf16(name, t, shape)
    _check_lse(lse, shape)
    B, H, N, d = shape
    lib = load()
    check("fa_fwd", lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               B, H, N, d, int(bool(causal)), float(scale), _stream_handle(stream)))


def _gqa_dims(q, k):
    """(B, Hq, Hkv, N, d) for q [B, Hq, N, d] and k [B, Hkv, N, d]."""
    B, Hq, N, d = _dims(q)
    if k.dim() != 4 or k.shape[0] != B or tuple(k.shape[2:]) != (N, d):
        raise ValueError("k must be [B, Hkv, N, d] with q's B, N, d")
    Hkv = int(k.shape[1])
    if Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"the query heads ({Hq}) must be a multiple of the K/V heads ({Hkv})")
    return B, Hq, Hkv, N, d


def fa_fwd_gqa(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """fa_fwd_gqa of the C ABI: q, o [B, Hq, N, d]; k, v [B, Hkv, N, d]; lse [B, Hq, N]."""
    B, Hq, Hkv, N, d = _gqa_dims(q, k)
    for name, t, shape in (("q", q, (B, Hq, N, d)), ("k", k, (B, Hkv, N, d)), ("v", v, (B, Hkv, N, d)),
                           ("o", o, (B, Hq, N, d))):
        _check_bf16(name, t, shape)
    _check_lse(lse, (B, Hq, N, d))
    lib = load()
    check("fa_fwd_gqa", lib.fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                       B, Hq, Hkv, N, d, int(bool(causal)), float(scale), _stream_handle(stream)))


def fa_bwd_gqa(q, k, v, o, lse, do, dq, dk, dv, causal: bool, scale: float, workspace, stream=None) -> None:
    """fa_bwd_gqa of the C ABI: q, o, do, dq [B, Hq, N, d]; k, v, dk, dv [B, Hkv, N, d].

    `workspace` is a CUDA uint8 tensor of at least fa_bwd_workspace_size(B, Hq, N, d) bytes.
    """
    B, Hq, Hkv, N, d = _gqa_dims(q, k)
    qs, ks = (B, Hq, N, d), (B, Hkv, N, d)
    for name, t, shape in (("q", q, qs), ("k", k, ks), ("v", v, ks), ("o", o, qs), ("do", do, qs), ("dq", dq, qs),
                           ("dk", dk, ks), ("dv", dv, ks)):
        _check_bf16(name, t, shape)
    _check_lse(lse, qs)
    lib = load()
    check("fa_bwd_gqa", lib.fa_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                       do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                       B, Hq, Hkv, N, d, int(bool(causal)), float(scale), *_ws(workspace),
                                       _stream_handle(stream)))


def fa_fwd_splitkv_workspace_size(B: int, Hq: int, Nq: int, d: int, num_splits: int) -> int:
    return int(load().fa_fwd_splitkv_workspace_size(B, Hq, Nq, d, num_splits))


def fa_fwd_splitkv(q, k, v, o, lse, causal: bool, scale: float, num_splits: int = 0, workspace=None,
                   stream=None) -> None:
    """fa_fwd_splitkv of the C ABI: q, o [B, Hq, Nq, d]; k, v [B, Hkv, Nk, d]; lse [B, Hq, Nq].

    Causal masks align to the last key (query i sees keys j <= i + Nk - Nq).
    num_splits = 0 lets the library choose within `workspace` (a CUDA uint8
    tensor, or None for no split).
    """
    B, Hq, Nq, d = _dims(q)
    if k.dim() != 4 or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k must be [B, Hkv, Nk, d] with q's B and d")
    Hkv, Nk = int(k.shape[1]), int(k.shape[2])
    for name, t, shape in (("q", q, (B, Hq, Nq, d)), ("k", k, (B, Hkv, Nk, d)), ("v", v, (B, Hkv, Nk, d)),
                           ("o", o, (B, Hq, Nq, d))):
        _check_bf16(name, t, shape)
    _check_lse(lse, (B, Hq, Nq, d))
    check("fa_fwd_splitkv", load().fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                                  lse.data_ptr(), B, Hq, Hkv, Nq, Nk, d, int(bool(causal)),
                                                  float(scale), int(num_splits), *_ws(workspace),
                                                  _stream_handle(stream)))


def fa_bwd_deterministic(q, k, v, o, lse, do, dq, dk, dv, causal: bool, scale: float, workspace, stream=None) -> None:
    """fa_bwd_deterministic of the C ABI: fa_bwd with a bitwise-reproducible dq (d = 64, 128)."""
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bf16(name, t, shape)
    _check_lse(lse, shape)
    B, H, N, d = shape
    check("fa_bwd_deterministic",
          load().fa_bwd_deterministic(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                      do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                                      int(bool(causal)), float(scale), *_ws(workspace), _stream_handle(stream)))


def fa_bwd_gqa_deterministic(q, k, v, o, lse, do, dq, dk, dv, causal: bool, scale: float, workspace,
                             stream=None) -> None:
    """fa_bwd_gqa_deterministic of the C ABI: fa_bwd_gqa with a bitwise-reproducible dq (d = 64, 128)."""
    B, Hq, Hkv, N, d = _gqa_dims(q, k)
    qs, ks = (B, Hq, N, d), (B, Hkv, N, d)
    for name, t, shape in (("q", q, qs), ("k", k, ks), ("v", v, ks), ("o", o, qs), ("do", do, qs), ("dq", dq, qs),
                           ("dk", dk, ks), ("dv", dv, ks)):
        _check_bf16(name, t, shape)
    _check_lse(lse, qs)
    check("fa_bwd_gqa_deterministic",
          load().fa_bwd_gqa_deterministic(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                          do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv,
                                          N, d, int(bool(causal)), float(scale), *_ws(workspace),
                                          _stream_handle(stream)))


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd_gqa_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load().fa_bwd_gqa_workspace_size(B, Hq, Hkv, N, d))


def fa_bwd(q, k, v, o, lse, do, dq, dk, dv, causal: bool, scale: float, workspace, stream=None) -> None:
    """fa_bwd of the C ABI on torch tensors (dq, dk, dv written in place).

    `workspace` is a CUDA uint8 tensor of at least fa_bwd_workspace_size() bytes.
    """
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bf16(name, t, shape)
    _check_lse(lse, shape)
    B, H, N, d = shape
    lib = load()
    check("fa_bwd", lib.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                               B, H, N, d, int(bool(causal)), float(scale), *_ws(workspace),
                               _stream_handle(stream)))


def _ws(workspace):
    if workspace is None:
        return 0, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fa_bwd_preprocess(o, lse, do, workspace, stream=None) -> None:
    """First phase of fa_bwd: D, base-2 L and a zeroed dQ accumulator in `workspace`."""
    shape = _dims(o)
    _check_bf16("o", o, shape)
    _check_bf16("do", do, shape)
    _check_lse(lse, shape)
    B, H, N, d = shape
    check("fa_bwd_preprocess", load().fa_bwd_preprocess(o.data_ptr(), lse.data_ptr(), do.data_ptr(), B, H, N, d,
                                                        *_ws(workspace), _stream_handle(stream)))


def fa_bwd_preprocess_stats(o, lse, do, workspace, stream=None) -> None:
    """First phase of fa_bwd_deterministic: D and base-2 L in `workspace` (no accumulator zeroing)."""
    shape = _dims(o)
    _check_bf16("o", o, shape)
    _check_bf16("do", do, shape)
    _check_lse(lse, shape)
    B, H, N, d = shape
    check("fa_bwd_preprocess_stats", load().fa_bwd_preprocess_stats(o.data_ptr(), lse.data_ptr(), do.data_ptr(), B,
                                                                    H, N, d, *_ws(workspace), _stream_handle(stream)))


def fa_bwd_main(q, k, v, do, dk, dv, causal: bool, scale: float, workspace, stream=None) -> None:
    """Second phase of fa_bwd: dk, dv, and dQ accumulated into `workspace`."""
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do), ("dk", dk), ("dv", dv)):
        _check_bf16(name, t, shape)
    B, H, N, d = shape
    check("fa_bwd_main", load().fa_bwd_main(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), dk.data_ptr(),
                                            dv.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                            *_ws(workspace), _stream_handle(stream)))


def fa_bwd_dkdv(q, k, v, do, dk, dv, causal: bool, scale: float, workspace, stream=None) -> None:
    """Deterministic backward phase: dk, dv only (after fa_bwd_preprocess)."""
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do), ("dk", dk), ("dv", dv)):
        _check_bf16(name, t, shape)
    B, H, N, d = shape
    check("fa_bwd_dkdv", load().fa_bwd_dkdv(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), dk.data_ptr(),
                                            dv.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                            *_ws(workspace), _stream_handle(stream)))


def fa_bwd_dq(q, k, v, do, dq, causal: bool, scale: float, workspace, stream=None) -> None:
    """Deterministic backward phase: dq summed per query tile on chip (after fa_bwd_preprocess)."""
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do), ("dq", dq)):
        _check_bf16(name, t, shape)
    B, H, N, d = shape
    check("fa_bwd_dq", load().fa_bwd_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), dq.data_ptr(),
                                        B, H, N, d, int(bool(causal)), float(scale), *_ws(workspace),
                                        _stream_handle(stream)))


def fa_bwd_postprocess(dq, workspace, stream=None) -> None:
    """Last phase of fa_bwd: dq = bf16(dQ accumulator)."""
    shape = _dims(dq)
    _check_bf16("dq", dq, shape)
    B, H, N, d = shape
    check("fa_bwd_postprocess", load().fa_bwd_postprocess(dq.data_ptr(), B, H, N, d, *_ws(workspace),
                                                          _stream_handle(stream)))


# Scratch size compiled into the library for fa_bwd_noalloc (include/fa.h).
FA_BWD_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def fa_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, causal: bool, scale: float, stream=None) -> None:
    """fa_bwd without a caller workspace: the library's fixed scratch array is used.

    For callers that are given only input and output buffers and cannot
    allocate device memory. Sizes whose workspace exceeds
    FA_BWD_NOALLOC_SCRATCH_BYTES raise FAError(FA_ERR_WORKSPACE). Calls that
    overlap on the GPU share the array and race.
    """
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bf16(name, t, shape)
    _check_lse(lse, shape)
    B, H, N, d = shape
    check("fa_bwd_noalloc", load().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                                  lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                                  dv.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                                  _stream_handle(stream)))


def fa_fwd_bwd_host_device_bytes(B: int, H: int, N: int, d: int) -> int:
    """Device buffer size fa_fwd_bwd_host needs (0 for invalid or empty problems)."""
    return int(load().fa_fwd_bwd_host_device_bytes(B, H, N, d))


def _check_host(name, t, shape, dtype):
    if t.dtype != dtype or tuple(t.shape) != shape or t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CPU tensor of shape {shape}")


# Host tensors of calls in flight. torch hands a page-locked tensor that the
# caller has dropped out again at once: it knows nothing of the library's copies.
_in_flight = []
_in_flight_lock = threading.Lock()


def _drop_finished() -> None:
    with _in_flight_lock:
        _in_flight[:] = [call for call in _in_flight if not call[0].query()]


def _hold(stream, *tensors) -> None:
    """Keep a call's host tensors until the stream has done its work (looked at by the next such call and
    by fa_get_device_status). A captured call's tensors are the caller's to keep, as long as the graph."""
    import torch
    with _on_stream(stream):
        if torch.cuda.is_current_stream_capturing():
            return
        event = torch.cuda.Event()
        event.record()
    _drop_finished()
    with _in_flight_lock:
        _in_flight.append((event, tensors))


def fa_fwd_bwd_host(q, k, v, do, o, lse, dq, dk, dv, causal: bool, scale: float, device_buffer,
                    stream=None) -> None:
    """fa_fwd_bwd_host of the C ABI: forward and backward of CPU tensors.

    q, k, v, do (in) and o, dq, dk, dv (out) are contiguous bf16 CPU tensors
    [B, H, N, d], lse a float32 CPU tensor [B, H, N]; page-locked tensors
    (pin_memory) let the library overlap the copies with the kernels.
    device_buffer is a CUDA uint8 tensor of at least
    fa_fwd_bwd_host_device_bytes(B, H, N, d) bytes. Asynchronous on `stream`:
    the outputs are valid once the stream has synchronised. The host tensors
    may be dropped before that, but not written to.
    """
    import torch
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do), ("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_host(name, t, shape, torch.bfloat16)
    _check_host("lse", lse, shape[:3], torch.float32)
    if not device_buffer.is_cuda or device_buffer.dtype != torch.uint8:
        raise ValueError("device_buffer must be a CUDA uint8 tensor")
    B, H, N, d = shape
    check("fa_fwd_bwd_host", load().fa_fwd_bwd_host(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), o.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), B, H, N, d, int(bool(causal)), float(scale), device_buffer.data_ptr(),
        device_buffer.numel(), _stream_handle(stream)))
    _hold(stream, q, k, v, do, o, lse, dq, dk, dv)


def fa_fwd_host_device_bytes(B: int, H: int, N: int, d: int) -> int:
    """Device buffer size fa_fwd_host needs (0 for invalid or empty problems)."""
    return int(load().fa_fwd_host_device_bytes(B, H, N, d))


def fa_fwd_host(q, k, v, o, lse, causal: bool, scale: float, device_buffer, stream=None) -> None:
    """fa_fwd_host of the C ABI: the forward of CPU tensors, pipelined over head chunks.

    q, k, v (in) and o (out) are contiguous bf16 CPU tensors [B, H, N, d], lse
    a float32 CPU tensor [B, H, N]; device_buffer a CUDA uint8 tensor of at
    least fa_fwd_host_device_bytes(B, H, N, d) bytes. Asynchronous on `stream`.
    """
    import torch
    shape = _dims(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check_host(name, t, shape, torch.bfloat16)
    _check_host("lse", lse, shape[:3], torch.float32)
    if not device_buffer.is_cuda or device_buffer.dtype != torch.uint8:
        raise ValueError("device_buffer must be a CUDA uint8 tensor")
    B, H, N, d = shape
    check("fa_fwd_host", load().fa_fwd_host(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d, int(bool(causal)),
        float(scale), device_buffer.data_ptr(), device_buffer.numel(), _stream_handle(stream)))
    _hold(stream, q, k, v, o, lse)


def rope_tables(rows: int, rot: int, base: float = 10000.0, device="cuda"):
    """Cosines and sines of the position rotation, fp32 [rows, rot / 2] each: the
    angle of pair i at position p is p * base^(-2 i / rot), formed in 64 bits."""
    import torch
    freq = torch.pow(torch.tensor(base, dtype=torch.float64),
                     -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq.to(device)[None, :]
    return angle.cos().float(), angle.sin().float()


# The wrappers below are called once per layer and token, so their checks are
# written for the call that passes them: one expression over the tensors'
# attributes. Only a call that fails it is looked at tensor by tensor, for its
# message.
def _refuse(named):
    """Raise for the first of (name, tensor, dtypes, shape, contiguous) that is not as it should be."""
    import torch
    for name, t, dtypes, shape, contiguous in named:
        if t is None:
            continue
        if t.dtype not in dtypes:  # as for the other entry points: TypeError for values, ValueError for the rest
            values = torch.bfloat16 in dtypes or torch.uint8 in dtypes or torch.float8_e4m3fn in dtypes
            raise (TypeError if values else ValueError)(f"{name} must be {' or '.join(str(x)[6:] for x in dtypes)}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}'s last dimension must be contiguous")
    here = torch.cuda.current_device()
    for name, t, *_ in named:
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name} must be on the current CUDA device (cuda:{here}), got {t.device}")
    raise ValueError("tensors of one call must have matching types, shapes and devices")


def _bytes(workspace):
    """Is the workspace, if given, one run of bytes?"""
    import torch
    return workspace is None or (workspace.dtype == torch.uint8 and workspace.is_contiguous())


def _devices(*tensors):
    """Their CUDA devices (None for a tensor not given; -1: not on a GPU)."""
    return {t.get_device() for t in tensors if t is not None}


_Strides = ctypes.c_longlong * 9
_NO_STRIDES = (0, 0, 0, 1)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _norm_rope_named(B, Hq, Hkv, N, d, qkv, strided, w, cos, sin, positions, dw, workspace):
    import torch
    bf, f32 = (torch.bfloat16,), (torch.float32,)
    qs, ks = (B, Hq, N, d), (B, Hkv, N, d)
    named = [(n, t, bf, s, True) for (n, t), s in zip(qkv, (qs, ks, ks))]
    named += [(n, t, bf, qs if n.lstrip("d")[0] == "q" else ks, False) for n, t in strided]
    named += [(n, t, (torch.float32, torch.bfloat16) if w[0][1] is None else (w[0][1].dtype,), (d,), True) for n, t in w]
    if cos is not None:
        named += [(n, t, f32, cos.shape, True) for n, t in (("cos", cos), ("sin", sin))]
    named += [(n, t, f32, (d,), True) for n, t in dw]
    if positions is not None:
        named.append(("positions", positions, (torch.int32,), (B, N), True))
    if workspace is not None:
        named.append(("workspace", workspace, (torch.uint8,), workspace.shape, True))
    return named


def _norm_rope_tables(wq, wk, cos, sin):
    """The weights' type flag, the tables' rows and rot."""
    import torch
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk are given together or not at all")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin are given together or not at all")
    w_bf16 = 0
    if wq is not None:
        if wq.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"wq must be float32 or bfloat16, got {wq.dtype}")
        w_bf16 = int(wq.dtype == torch.bfloat16)
    if cos is None:
        return w_bf16, 0, 0
    if cos.dim() != 2:
        raise ValueError("cos and sin must be [rows, rot / 2] tensors")
    rows, half = cos.shape
    return w_bf16, rows, 2 * half


def _norm_rope_ok(wq, wk, cos, sin, positions, B, N, d):
    """Are the tensors the two directions share as they should be?"""
    import torch
    return ((wq is None or (wk.dtype == wq.dtype and wq.shape == wk.shape == (d,) and wq.is_contiguous()
                            and wk.is_contiguous()))
            and (cos is None or (cos.dtype == sin.dtype == torch.float32 and cos.shape == sin.shape
                                 and cos.is_contiguous() and sin.is_contiguous()))
            and (positions is None or (positions.dtype == torch.int32 and positions.shape == (B, N)
                                       and positions.is_contiguous())))


def fa_norm_rope_fwd(q_in, k_in, v_in, wq, wk, cos, sin, positions, q, k, v, interleaved: bool = False,
                     eps: float = 1e-6, stream=None) -> None:
    """fa_norm_rope_fwd of the C ABI: q_in [B, Hq, N, d], k_in, v_in [B, Hkv, N, d] with any
    strides and contiguous rows (views of a packed projection); q, k, v contiguous.

    wq, wk None: no norm. cos, sin (rope_tables) None: no rotation. v_in, v
    None: no values. positions None: token n is at position n.
    """
    import torch
    bf = torch.bfloat16
    qs, ks = q_in.shape, k_in.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    if (v_in is None) != (v is None):
        raise ValueError("v_in and v are given together or not at all")
    B, Hq, N, d = qs
    Hkv = ks[1]
    w_bf16, rows, rot = _norm_rope_tables(wq, wk, cos, sin)
    sq, sk, sv = q_in.stride(), k_in.stride(), _NO_STRIDES if v_in is None else v_in.stride()
    if not (q_in.dtype == k_in.dtype == q.dtype == k.dtype == bf and q.shape == qs and k.shape == ks
            and ks == (B, Hkv, N, d) and sq[3] == sk[3] == 1 and q.is_contiguous() and k.is_contiguous()
            and (v is None or (v_in.dtype == v.dtype == bf and v_in.shape == v.shape == ks and sv[3] == 1
                               and v.is_contiguous()))
            and _norm_rope_ok(wq, wk, cos, sin, positions, B, N, d)
            and _devices(q_in, k_in, v_in, wq, wk, cos, sin, positions, q, k, v) == {torch.cuda.current_device()}):
        _refuse(_norm_rope_named(B, Hq, Hkv, N, d, (("q", q), ("k", k), ("v", v)),
                                 (("q_in", q_in), ("k_in", k_in), ("v_in", v_in)), (("wq", wq), ("wk", wk)), cos, sin,
                                 positions, (), None))
    check("fa_norm_rope_fwd", load().fa_norm_rope_fwd(
        q_in.data_ptr(), k_in.data_ptr(), _ptr(v_in), _Strides(*sq[:3], *sk[:3], *sv[:3]), _ptr(wq), _ptr(wk), w_bf16,
        _ptr(cos), _ptr(sin), rows, _ptr(positions), q.data_ptr(), k.data_ptr(), _ptr(v), B, Hq, Hkv, N, d, rot,
        1 if interleaved else 0, eps, _stream_handle(stream)))


def fa_norm_rope_bwd_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load().fa_norm_rope_bwd_workspace_size(B, Hq, Hkv, N, d))


def fa_norm_rope_bwd(dq, dk, dv, q_in, k_in, wq, wk, cos, sin, positions, dq_in, dk_in, dv_in, dwq, dwk, workspace,
                     interleaved: bool = False, eps: float = 1e-6, stream=None) -> None:
    """fa_norm_rope_bwd of the C ABI: dq [B, Hq, N, d], dk, dv [B, Hkv, N, d] contiguous (in); q_in,
    k_in as in the forward; dq_in, dk_in, dv_in (out) with any strides that keep
    their rows apart; dwq, dwk float32 [d] (out).

    Without weights q_in, k_in, dwq, dwk and workspace are not used.
    """
    import torch
    bf = torch.bfloat16
    qs, ks = dq.shape, dk.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    if (dv is None) != (dv_in is None):
        raise ValueError("dv and dv_in are given together or not at all")
    B, Hq, N, d = qs
    Hkv = ks[1]
    w_bf16, rows, rot = _norm_rope_tables(wq, wk, cos, sin)
    if wq is None:
        q_in = k_in = dwq = dwk = None
    sq, sk, sv = dq_in.stride(), dk_in.stride(), _NO_STRIDES if dv is None else dv_in.stride()
    xq, xk = (_NO_STRIDES, _NO_STRIDES) if wq is None else (q_in.stride(), k_in.stride())
    if not (dq.dtype == dk.dtype == dq_in.dtype == dk_in.dtype == bf and dq_in.shape == qs and dk_in.shape == ks
            and ks == (B, Hkv, N, d) and sq[3] == sk[3] == 1 and dq.is_contiguous() and dk.is_contiguous()
            and (dv is None or (dv_in.dtype == dv.dtype == bf and dv_in.shape == dv.shape == ks and sv[3] == 1
                                and dv.is_contiguous()))
            and (wq is None or (q_in.dtype == k_in.dtype == bf and q_in.shape == qs and k_in.shape == ks
                                and xq[3] == xk[3] == 1 and dwq.dtype == dwk.dtype == torch.float32
                                and dwq.shape == dwk.shape == (d,) and dwq.is_contiguous() and dwk.is_contiguous()))
            and _norm_rope_ok(wq, wk, cos, sin, positions, B, N, d)
            and _bytes(workspace)
            and _devices(dq, dk, dv, q_in, k_in, wq, wk, cos, sin, positions, dq_in, dk_in, dv_in, dwq, dwk,
                         workspace) == {torch.cuda.current_device()}):
        _refuse(_norm_rope_named(B, Hq, Hkv, N, d, (("dq", dq), ("dk", dk), ("dv", dv)),
                                 (("dq_in", dq_in), ("dk_in", dk_in), ("dv_in", dv_in), ("q_in", q_in), ("k_in", k_in)),
                                 (("wq", wq), ("wk", wk)), cos, sin, positions, (("dwq", dwq), ("dwk", dwk)), workspace))
    check("fa_norm_rope_bwd", load().fa_norm_rope_bwd(
        dq.data_ptr(), dk.data_ptr(), _ptr(dv), _ptr(q_in), _ptr(k_in), _Strides(*xq[:3], *xk[:3]), _ptr(wq), _ptr(wk),
        w_bf16, _ptr(cos), _ptr(sin), rows, _ptr(positions), dq_in.data_ptr(), dk_in.data_ptr(), _ptr(dv_in),
        _Strides(*sq[:3], *sk[:3], *sv[:3]), _ptr(dwq), _ptr(dwk), B, Hq, Hkv, N, d, rot, 1 if interleaved else 0, eps,
        *_ws(workspace), _stream_handle(stream)))


def _kv8_dims(k_cache, v_cache, k_scale, v_scale, page_table, lens, counts, *rows):
    """Checks of a paged 8-bit cache and of the call's own bf16 tensors (name, tensor, heads,
    tokens); returns (B, Hkv, d, page, num_pages, max_pages)."""
    import torch
    shape, B_pages = k_cache.shape, page_table.shape
    if len(shape) != 4 or len(B_pages) != 2:
        raise ValueError("k_cache must be [num_pages, Hkv, page, d] and page_table [B, max_pages]")
    pages, Hkv, page, d = shape
    B, max_pages = B_pages
    i32, per_head = torch.int32, (pages, Hkv)
    tensors = [t for _, t, _, _ in rows]
    if not (v_cache.dtype == k_cache.dtype and v_cache.shape == shape and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_cache.dtype in (torch.uint8, torch.float8_e4m3fn)
            and k_scale.dtype == v_scale.dtype == torch.float32 and k_scale.shape == v_scale.shape == per_head
            and k_scale.is_contiguous() and v_scale.is_contiguous()
            and page_table.dtype == lens.dtype == i32 and page_table.is_contiguous() and lens.shape == (B,)
            and lens.is_contiguous()
            and (counts is None or (counts.dtype == i32 and counts.shape == (B,) and counts.is_contiguous()))
            and all([t.dtype == torch.bfloat16 and t.shape == (B, heads, n, d) and t.is_contiguous()
                     for _, t, heads, n in rows])
            and _devices(k_cache, v_cache, k_scale, v_scale, page_table, lens, counts, *tensors)
            == {torch.cuda.current_device()}):
        code = (torch.uint8, torch.float8_e4m3fn)
        _refuse([("k_cache", k_cache, code, shape, True), ("v_cache", v_cache, (k_cache.dtype,), shape, True),
                 ("k_scale", k_scale, (torch.float32,), per_head, True),
                 ("v_scale", v_scale, (torch.float32,), per_head, True),
                 ("page_table", page_table, (i32,), B_pages, True), ("lens", lens, (i32,), (B,), True),
                 ("counts", counts, (i32,), (B,), True)]
                + [(name, t, (torch.bfloat16,), (B, heads, n, d), True) for name, t, heads, n in rows])
    return B, Hkv, d, page, pages, max_pages


def fa_kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, lens, counts=None, stream=None) -> None:
    """fa_kv8_append of the C ABI: quantise k, v [B, Hkv, n, d] (bf16, contiguous) into the pages of
    the last counts[b] (None: n) of lens[b] tokens of each sequence.

    k_cache, v_cache: uint8 or float8_e4m3fn [num_pages, Hkv, page, d]; k_scale,
    v_scale float32 [num_pages, Hkv]; page_table int32 [B, max_pages]; lens,
    counts int32 [B].
    """
    if k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    n, heads = k.shape[2], k_cache.shape[1]
    B, Hkv, d, page, pages, max_pages = _kv8_dims(k_cache, v_cache, k_scale, v_scale, page_table, lens, counts,
                                                  ("k", k, heads, n), ("v", v, heads, n))
    check("fa_kv8_append", load().fa_kv8_append(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        page_table.data_ptr(), lens.data_ptr(), _ptr(counts), B, Hkv, n, d, page, pages, max_pages,
        _stream_handle(stream)))


def fa_kv8_advance(lens, counts, taken, n: int, page: int, max_pages: int, stream=None) -> None:
    """fa_kv8_advance of the C ABI: lens[b] += counts[b] (None: n) where the sequence can take them, with
    taken[b] the tokens it takes: what fa_kv8_append then needs as its counts. int32 [B] each."""
    import torch
    i32, shape = torch.int32, lens.shape
    if not (lens.dtype == taken.dtype == i32 and len(shape) == 1 and taken.shape == shape and lens.is_contiguous()
            and taken.is_contiguous()
            and (counts is None or (counts.dtype == i32 and counts.shape == shape and counts.is_contiguous()))
            and _devices(lens, counts, taken) == {torch.cuda.current_device()}):
        if len(shape) != 1:
            raise ValueError("lens must be an int32 [B] tensor")
        _refuse([(name, t, (i32,), shape, True) for name, t in (("lens", lens), ("counts", counts), ("taken", taken))])
    check("fa_kv8_advance", load().fa_kv8_advance(lens.data_ptr(), _ptr(counts), taken.data_ptr(), shape[0], n, page,
                                                  max_pages, _stream_handle(stream)))


def fa_kv8_gather(k_cache, v_cache, k_scale, v_scale, page_table, lens, k, v, stream=None) -> None:
    """fa_kv8_gather of the C ABI: rows [0, min(lens[b], n)) of each sequence back as bf16 into
    k, v [B, Hkv, n, d]; later rows are left as they were."""
    if k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    n, heads = k.shape[2], k_cache.shape[1]
    B, Hkv, d, page, pages, max_pages = _kv8_dims(k_cache, v_cache, k_scale, v_scale, page_table, lens, None,
                                                  ("k", k, heads, n), ("v", v, heads, n))
    check("fa_kv8_gather", load().fa_kv8_gather(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
        lens.data_ptr(), k.data_ptr(), v.data_ptr(), B, Hkv, n, d, page, pages, max_pages, _stream_handle(stream)))


def fa_fwd_kv8_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    return int(load().fa_fwd_kv8_workspace_size(B, Hq, Hkv, Nq, d))


def fa_fwd_kv8(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, o, lse, causal: bool, scale: float,
               counts=None, workspace=None, stream=None) -> None:
    """fa_fwd_kv8 of the C ABI: attention of q [B, Hq, Nq, d] over the paged 8-bit cache into o (like
    q) and lse float32 [B, Hq, Nq]; query i < counts[b] (None: Nq) stands at
    position lens[b] - counts[b] + i of its sequence.

    workspace is a CUDA uint8 tensor of at least fa_fwd_kv8_workspace_size() bytes.
    """
    _fwd_kv8("fa_fwd_kv8", q, k_cache, v_cache, k_scale, v_scale, page_table, lens, o, lse, causal, scale, counts,
             workspace, stream)


def fa_fwd_kv8_filled(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, o, lse, causal: bool, scale: float,
                      counts=None, workspace=None, stream=None) -> None:
    """fa_fwd_kv8_filled of the C ABI: fa_fwd_kv8, with zeros in the rows of o and lse that have no result (past
    counts[b], or of a sequence whose length or count is out of range)."""
    _fwd_kv8("fa_fwd_kv8_filled", q, k_cache, v_cache, k_scale, v_scale, page_table, lens, o, lse, causal, scale, counts,
             workspace, stream)


def _fwd_kv8(name, q, k_cache, v_cache, k_scale, v_scale, page_table, lens, o, lse, causal, scale, counts, workspace,
             stream):
    import torch
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    _, Hq, Nq, _ = q.shape
    B, Hkv, d, page, pages, max_pages = _kv8_dims(k_cache, v_cache, k_scale, v_scale, page_table, lens, counts,
                                                  ("q", q, Hq, Nq), ("o", o, Hq, Nq))
    if Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"the query heads ({Hq}) must be a multiple of the K/V heads ({Hkv})")
    if not (lse.dtype == torch.float32 and lse.shape == (B, Hq, Nq) and lse.is_contiguous()
            and _bytes(workspace) and _devices(q, lse, workspace) == {q.get_device()}):
        _refuse((("lse", lse, (torch.float32,), (B, Hq, Nq), True),
                 ("workspace", workspace, (torch.uint8,), () if workspace is None else workspace.shape, True)))
    check(name, getattr(load(), name)(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        page_table.data_ptr(), lens.data_ptr(), _ptr(counts), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Nq, d, page,
        pages, max_pages, 1 if causal else 0, scale, *_ws(workspace), _stream_handle(stream)))


def fa_get_device_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device status (0 = FA_OK)."""
    st = int(load().fa_get_device_status(_stream_handle(stream)))
    _drop_finished()
    return st


def fa_get_device_status_detail(stream=None) -> tuple:
    """Synchronise the stream; return and clear the whole device status word:
    (code, role of the first wait that gave up, its block, its thread)."""
    word = (ctypes.c_uint * 4)()
    st = int(load().fa_get_device_status_detail(ctypes.addressof(word), _stream_handle(stream)))
    _drop_finished()
    if st == 7:  # FA_ERR_CUDA: the synchronisation failed, the word was not read
        check("fa_get_device_status_detail", st)
    return tuple(int(x) for x in word)


def fa_set_wait_limit_ns(limit_ns: int) -> None:
    load().fa_set_wait_limit_ns(int(limit_ns))


def fa_debug_timeout_probe(limit_ns: int, stream=None) -> None:
    check("fa_debug_timeout_probe", load().fa_debug_timeout_probe(int(limit_ns), _stream_handle(stream)))


def fa_debug_skip_arrival(role: int) -> None:
    """Test hook: block 0 of later launches leaves out the first arrival of
    `role` (a role code of fa_get_device_status_detail), so a bounded wait
    gives up; 0 turns it off."""
    check("fa_debug_skip_arrival", load().fa_debug_skip_arrival(int(role)))


def forward(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Allocate O (bf16) and L (fp32) with torch and run fa_fwd (fa_fwd_gqa when
    k, v have fewer heads than q)."""
    import torch
    B, H, N, d = _dims(q)
    if scale is None:
        scale = default_scale(d)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if k.dim() == 4 and k.shape[1] != H:
        fa_fwd_gqa(q, k, v, o, lse, causal, scale, stream)
    else:
        fa_fwd(q, k, v, o, lse, causal, scale, stream)
    return o, lse


def backward(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, workspace=None, stream=None,
             deterministic: bool = False):
    """Allocate dQ, dK, dV (and the workspace if not given) with torch and run fa_bwd
    (fa_bwd_gqa when k, v have fewer heads than q; the *_deterministic entry
    points when `deterministic`)."""
    import torch
    B, H, N, d = _dims(q)
    if scale is None:
        scale = default_scale(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    grouped = k.dim() == 4 and k.shape[1] != H
    if workspace is None:
        size = fa_bwd_gqa_workspace_size(B, H, int(k.shape[1]), N, d) if grouped else fa_bwd_workspace_size(B, H, N, d)
        workspace = torch.empty(max(1, size), dtype=torch.uint8, device=q.device)
    if grouped:
        fn = fa_bwd_gqa_deterministic if deterministic else fa_bwd_gqa
    else:
        fn = fa_bwd_deterministic if deterministic else fa_bwd
    fn(q, k, v, o, lse, do, dq, dk, dv, causal, scale, workspace, stream)
    return dq, dk, dv


def norm_rope(q_in, k_in, v_in=None, wq=None, wk=None, cos=None, sin=None, positions=None, interleaved: bool = False,
              eps: float = 1e-6, stream=None):
    """Allocate q, k (and v) as [B, H, N, d] with torch and run fa_norm_rope_fwd: what `forward` and
    the cache take, from the views of a packed projection."""
    import torch
    with _on_stream(stream):
        q, k = (torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) for x in (q_in, k_in))
        v = None if v_in is None else torch.empty(v_in.shape, dtype=torch.bfloat16, device=v_in.device)
    fa_norm_rope_fwd(q_in, k_in, v_in, wq, wk, cos, sin, positions, q, k, v, interleaved, eps, stream)
    return q, k, v


def norm_rope_backward(dq, dk, dv, q_in, k_in, wq=None, wk=None, cos=None, sin=None, positions=None, out=None,
                       interleaved: bool = False, eps: float = 1e-6, workspace=None, stream=None):
    """Run fa_norm_rope_bwd on `backward`'s dq, dk, dv; returns (dq_in, dk_in, dv_in, dwq, dwk).

    out: (dq_in, dk_in, dv_in) to write, e.g. the views of one packed gradient;
    None allocates contiguous ones. dwq, dwk are float32 (None without weights).
    """
    import torch
    B, Hq, N, d = _dims(dq)
    dwq = dwk = None
    with _on_stream(stream):
        if out is None:
            out = (torch.empty_like(dq), torch.empty_like(dk), None if dv is None else torch.empty_like(dv))
        if wq is not None:
            dwq, dwk = (torch.empty(d, dtype=torch.float32, device=dq.device) for _ in range(2))
            if workspace is None:
                workspace = torch.empty(max(1, fa_norm_rope_bwd_workspace_size(B, Hq, int(dk.shape[1]), N, d)),
                                        dtype=torch.uint8, device=dq.device)
    fa_norm_rope_bwd(dq, dk, dv, q_in, k_in, wq, wk, cos, sin, positions, *out, dwq, dwk, workspace, interleaved, eps,
                     stream)
    return (*out, dwq, dwk)


def _on_stream(stream):
    """torch's context for a stream given as None, a torch stream or a raw handle: what is allocated
    in it may be freed while that stream still uses it."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class KV8Cache:
    """A paged 8-bit key/value cache of B sequences and the calls that use it.

    Holds the pools, scales, page table (each sequence's pages one after another
    unless `page_table` and `num_pages` are given) and lengths, all on the device:
    a decoding step (`append`, `attend`) can be captured into a CUDA graph. `lens` may be
    set by the caller, to values from 0 to max_pages * page.
    """

    def __init__(self, B: int, Hkv: int, d: int, max_tokens: int, page: int = 64, page_table=None, num_pages=None,
                 device="cuda"):
        import torch
        max_pages = -(-max_tokens // page)
        if page_table is None:
            num_pages = B * max_pages
            page_table = torch.arange(num_pages, dtype=torch.int32, device=device).view(B, max_pages)
        elif num_pages is None:
            raise ValueError("num_pages is needed with a page_table of your own")
        self.page_table = page_table
        self.k_cache, self.v_cache = (torch.empty(num_pages, Hkv, page, d, dtype=torch.uint8, device=device)
                                      for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones(num_pages, Hkv, dtype=torch.float32, device=device) for _ in range(2))
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self._taken = torch.zeros_like(self.lens)
        self._workspaces = {}

    def _cache(self):
        return self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.page_table, self.lens

    def append(self, k, v, counts=None, stream=None) -> None:
        """Lengthen each sequence by counts[b] (None: n) tokens and write k, v [B, Hkv, n, d] there.

        A sequence that would outgrow its pages (max_tokens, rounded up to whole ones), or whose counts[b] is not
        from 0 to n, is left as it was: its tokens are dropped, and FA_ERR_INDEX
        is in the device status (fa_get_device_status). A call that is refused leaves all lengths as they were."""
        with _on_stream(stream):
            fa_kv8_advance(self.lens, counts, self._taken, int(k.shape[2]), self.k_cache.shape[2],
                           self.page_table.shape[1], stream)
            try:
                fa_kv8_append(k, v, *self._cache(), self._taken, stream)
            except Exception:
                self.lens.sub_(self._taken)
                raise

    def gather(self, n: int, stream=None):
        """The first n tokens' k, v as bf16 [B, Hkv, n, d], zero past a sequence's length."""
        import torch
        pages, Hkv, page, d = self.k_cache.shape
        with _on_stream(stream):
            k, v = (torch.zeros(self.lens.shape[0], Hkv, n, d, dtype=torch.bfloat16, device=self.lens.device)
                    for _ in range(2))
        fa_kv8_gather(*self._cache(), k, v, stream)
        return k, v

    def attend(self, q, causal: bool = True, scale: float | None = None, counts=None, stream=None):
        """O, L of q [B, Hq, Nq, d], whose last rows are the cache's newest tokens (fa_fwd_kv8). Rows
        that have no result are zero in both: those past counts[b], and those of a sequence whose length or
        count is out of range (FA_ERR_INDEX in the device status). One workspace per stream is kept, as large as the
        calls so far needed; a captured call has one of its own, in its graph's memory."""
        import torch
        B, Hq, Nq, d = _dims(q)
        handle = _stream_handle(stream)
        size = max(1, fa_fwd_kv8_workspace_size(B, Hq, int(self.k_cache.shape[1]), Nq, d))
        with _on_stream(stream):
            o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
            workspace = self._workspaces.get(handle)
            capturing = torch.cuda.is_current_stream_capturing()
            if workspace is None or workspace.numel() < size or capturing:
                workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
                if not capturing:
                    self._workspaces[handle] = workspace
        fa_fwd_kv8_filled(q, *self._cache(), o, lse, causal, default_scale(d) if scale is None else scale, counts,
                          workspace, handle)
        return o, lse


def flops(B: int, H: int, N: int, d: int, causal: bool, mode: str = "fwd") -> float:
    """Algorithmic FLOPs of the pages' benchmark convention.

    forward = 4 * N^2 * d * H (* B), halved under a causal mask; backward = 2.5x
    forward (five matmuls instead of two); fwd+bwd = 3.5x forward. (Reading note
    on papers.chlience.com, "结果 1"; paper-graph-ui summary, "Evaluation
    Methodology".)
    """
    f = 4.0 * B * H * N * N * d
    if causal:
        f *= 0.5
    mult = {"fwd": 1.0, "bwd": 2.5, "fwd_bwd": 3.5}[mode]
    return f * mult
