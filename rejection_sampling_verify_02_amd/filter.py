"""Sampling and filtered logits under temperature, top-k, min-p and top-p.

Thin binding over ``include/spec_filter.h`` (which has the policy, the row codes and the
limits).  ``spec_sample`` comes here when a call asks for more than one temperature and top-k:

    tokens, status = spec_sample(logits, u, 0.8, top_p=0.95)
    tokens, status = spec_sample(logits, u, temperature, top_k, top_p=top_p, min_p=min_p)  # [B] tensors

and ``spec_filter_logits`` gives verification the same policy: with target and draft filtered,

    target, _ = spec_filter_logits(target, 0.8, top_p=0.95)
    draft, _ = spec_filter_logits(draft, 0.8, top_p=0.95)
    accepted, tokens = spec_verify(target, draft, draft_tokens, u_accept, u_sample, 0.8)

both go through it.  Calls are enqueued on the current stream of the tensors' device, or on
``stream``, may be captured into a HIP graph, and take work memory from torch's allocator on that
stream, or ``workspace``.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import _each, load_library
from .cache import _code, _device, _elsewhere, _ints, _raise, _raw_stream, _too_large, _work

ROW_BAD_POLICY = -11


class _Policy(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float),
                ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p), ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


def sv_filter_workspace_bytes(rows: int, V: int, dtype: int) -> int:
    return int(load_library().sv_filter_workspace_bytes(rows, V, dtype))


_filter_bytes = lru_cache(maxsize=1024)(sv_filter_workspace_bytes)


def sv_filter_launch_plan(draw: bool) -> list[str]:
    return load_library().sv_filter_launch_plan(int(draw)).decode().split(";")


def _floats(t, name: str, shape: tuple, dev: int):
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _policy(temperature, top_k, top_p, min_p, shape: tuple, dev: int) -> _Policy:
    p = _Policy(1.0, 0, 1.0, 0.0)
    if _each(temperature):
        p.temperatures = _floats(temperature, "temperature", shape, dev)
    else:
        p.temperature = float(temperature)
    if _each(top_k):
        p.top_ks = _ints(top_k, "top_k", shape, dev)
    else:
        p.top_k = max(-1, min(int(top_k), 0x7FFFFFFF))  # any k beyond the vocabulary is none
    if _each(top_p):
        p.top_ps = _floats(top_p, "top_p", shape, dev)
    else:
        p.top_p = float(top_p)
    if _each(min_p):
        p.min_ps = _floats(min_p, "min_p", shape, dev)
    else:
        p.min_p = float(min_p)
    return p


def _space(workspace, rows: int, V: int, dt: int, dev: int):
    if workspace is not None and not isinstance(workspace, torch.Tensor):
        raise TypeError(f"workspace must be a uint8 tensor or None here, got {type(workspace).__name__}")
    return _work(workspace, _filter_bytes(rows, V, dt), dev)


def _events(events):
    return (None, 0) if events is None else ((ctypes.c_void_p * len(events))(*events), len(events))


def sample(logits, u, temperature, top_k, top_p, min_p, workspace, stream, out, events):
    """spec_sample's rows under the whole policy."""
    dev = _device(logits, "logits")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return sample(logits, u, temperature, top_k, top_p, min_p, workspace, None, out, events)
    dt = _code(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    B, V = logits.shape
    if B | V > 0x7FFFFFFF:
        _too_large("logits", B, V)
    rows = (B,)
    pol = _policy(temperature, top_k, top_p, min_p, rows, dev)
    up = None if u is None else _floats(u, "u", rows, dev)
    if out is not None:
        tok, st = out
        _ints(tok, "tokens", rows, dev), _ints(st, "row_status", rows, dev)
    else:
        tok, st = (torch.empty(rows, dtype=torch.int32, device=logits.device) for _ in range(2))
    ws = _space(workspace, B, V, dt, dev)
    ev, n_ev = _events(events)
    n = ctypes.c_int32(0)
    rc = load_library().spec_sample_filtered(logits.data_ptr(), dt, up, B, V, ctypes.byref(pol), tok.data_ptr(), st.data_ptr(), ws.data_ptr(),
                                             ws.numel(), _raw_stream(dev), ev, n_ev, ctypes.byref(n))
    if rc:
        _raise(rc)
    return (tok, st) if events is None else (tok, st, n.value)


def spec_filter_logits(logits, temperature, top_k=0, *, top_p=1.0, min_p=0.0, workspace=None, stream=None, out=None, events=None):
    """Logits [..., V] with -inf outside the set that the policy keeps (see include/spec_filter.h).
    temperature, top_k, top_p and min_p are numbers, or tensors of the leading shape (float32; top_k
    int32) with a setting for each row.  Returns (filtered [..., V], row_status [...] int32); ``out``
    may supply them, and filtered may be logits itself.  ``events`` as for spec_verify."""
    dev = _device(logits, "logits")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return spec_filter_logits(logits, temperature, top_k, top_p=top_p, min_p=min_p, workspace=workspace, out=out, events=events)
    dt = _code(logits, "logits")
    if logits.dim() < 1:
        raise ValueError("logits must be [..., V]")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    shape = logits.shape[:-1]
    V = logits.shape[-1]
    rows = shape.numel()
    if rows | V > 0x7FFFFFFF:
        _too_large("logits", rows, V)
    pol = _policy(temperature, top_k, top_p, min_p, shape, dev)
    if out is not None:
        to, st = out
        if to.dtype is not logits.dtype or to.shape != logits.shape or to.get_device() != dev or not to.is_contiguous():
            raise ValueError(f"out must be a contiguous {logits.dtype} tensor of shape {tuple(logits.shape)} on device {dev}")
        _ints(st, "row_status", shape, dev)
    else:
        to, st = torch.empty_like(logits), torch.empty(shape, dtype=torch.int32, device=logits.device)
    ws = _space(workspace, rows, V, dt, dev)
    ev, n_ev = _events(events)
    n = ctypes.c_int32(0)
    rc = load_library().spec_filter_logits(logits.data_ptr(), dt, rows, V, ctypes.byref(pol), to.data_ptr(), st.data_ptr(), ws.data_ptr(),
                                           ws.numel(), _raw_stream(dev), ev, n_ev, ctypes.byref(n))
    if rc:
        _raise(rc)
    return (to, st) if events is None else (to, st, n.value)
