"""The paged key-value cache of a speculative decoding round and the attention that reads it.

Thin binding over ``include/spec_cache.h`` (which has the layout, the semantics and the row
codes), in the manner of the verification's binding: arguments are checked and marshalled
here, every step runs in the library's HIP kernels, and nothing proceeds without the library.

    pool = PagePool.empty(num_pages, max_seqs, table_width, device)
    k_pages, v_pages = empty_pages(L, num_pages, Hkv, D, page_size, torch.bfloat16, device)
    room = spec_cache_resize(pool, cache_len, cache_len + N, k_pages, v_pages)
    for l in range(L):
        spec_cache_append(k, v, k_pages[l], v_pages[l], pool.page_table, cache_len, prior=room)
        out, status = spec_paged_attention(q, k_pages[l], v_pages[l], pool.page_table, cache_len, parent=parent, prior=room)
    acc, tokens, path = spec_tree_verify(target_logits, draft_logits, tokens, parent, ...)
    cache_len, status = spec_cache_commit(k_pages, v_pages, pool.page_table, cache_len, acc, path, prior=room)
    spec_cache_resize(pool, cache_len, cache_len, k_pages, v_pages)

``prior`` carries the resize's row codes on: a sequence that the pool had no pages left for may
still share its last page with others, and is left alone by the calls that would write to it.

Calls are enqueued on the current stream of the tensors' device, or on ``stream`` (a raw
hipStream_t), and may be captured into a HIP graph.  Work memory is taken for each call from
torch's allocator on that stream, so calls on different streams never share any; pass
``workspace`` (a uint8 tensor of at least the documented size) to keep it yourself.
"""
from __future__ import annotations

import ctypes
import math
from functools import lru_cache
from typing import NamedTuple

import torch

from . import SV_BF16, SV_F32, SpecVerifyError, load_library, sv_status_string

ROW_BAD_PAGE, ROW_BAD_LENGTH, ROW_NO_PAGES, ROW_BAD_FORK = -7, -8, -9, -10
CACHE_MAX_NEW, CACHE_MAX_SEQS = 1024, 4096
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


class PagePool(NamedTuple):
    """The books of a pool of pages: which sequence holds which, and which are free."""
    page_table: torch.Tensor  # [S, table_width] int32, -1 behind a sequence's pages
    seq_pages: torch.Tensor   # [S] int32 pages held
    ref_count: torch.Tensor   # [P] int32 sequences that hold a page
    free_map: torch.Tensor    # [ceil(P / 32)] int32, a bit for each page that nobody holds

    @classmethod
    def empty(cls, num_pages: int, max_seqs: int, table_width: int, device) -> "PagePool":
        i32 = dict(dtype=torch.int32, device=device)
        if num_pages < 1 or max_seqs < 1 or table_width < 1:
            raise ValueError(f"a pool has at least one page, sequence and table entry, got {num_pages}, {max_seqs}, {table_width}")
        free = torch.full(((num_pages + 31) // 32,), -1, **i32)
        if num_pages % 32:
            free[-1] = (1 << num_pages % 32) - 1
        return cls(torch.full((max_seqs, table_width), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(num_pages, **i32), free)


def empty_pages(layers: int, num_pages: int, kv_heads: int, head_dim: int, page_size: int, dtype, device):
    """Zeroed (k_pages, v_pages) of `layers` layers in the cache's layout."""
    if dtype not in (_BF16, _F32):
        raise TypeError(f"the cache must be bfloat16 or float32, got {dtype}")
    if head_dim < 16 or head_dim % 16 or not 16 <= page_size <= 256 or page_size & (page_size - 1):
        raise ValueError(f"head_dim must be a multiple of 16 and page_size a power of two from 16 to 256, got {head_dim} and {page_size}")
    E = 8 if dtype is _BF16 else 4
    return (torch.zeros((layers, num_pages, kv_heads, head_dim // E, page_size, E), dtype=dtype, device=device),
            torch.zeros((layers, num_pages, kv_heads, page_size // E, head_dim, E), dtype=dtype, device=device))


# The checks below take the usual case in one expression and look for the reason only when it
# fails: a call's host time is a few microseconds, and shows where its kernels take no longer.

_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _code(t: torch.Tensor, name: str) -> int:
    dt = t.dtype
    if dt is _BF16:
        return SV_BF16
    if dt is _F32:
        return SV_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {dt}")


def _int32(x: int, name: str) -> int:
    """x, if it is one: ctypes would pass its low 32 bits."""
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _too_large(name: str, *sizes):
    """The same for a tensor's sizes (an expanded one can have any), once one is found not to fit."""
    raise ValueError(f"{name}'s sizes must fit 32 bits, got {sizes}")


def _ints(t, name: str, shape: tuple, dev: int, optional: bool = False):
    """The address of a contiguous int32 tensor of that shape (None where it may be left out)."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{name} must be an int32 tensor, got None")
    if t.dtype is _I32 and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not _I32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _apart(outputs: dict, inputs: dict):
    """Outputs of the caller's that several workgroups write while others read those inputs."""
    for a, x in outputs.items():
        for b, y in inputs.items():
            if y is not None and x.data_ptr() < y.data_ptr() + 4 * y.numel() and y.data_ptr() < x.data_ptr() + 4 * x.numel():
                raise ValueError(f"{a} must not share memory with {b}")


def _pages(k_pages, v_pages, dims: int, dtype, dev: int):
    """(P, Hkv, D, page_size) of a cache of `dims` dimensions (5: a layer, 6: all of them)."""
    ks, vs = k_pages.shape, v_pages.shape
    E = 8 if dtype is _BF16 else 4
    if len(ks) == dims:
        *lead, U, page, e = ks
        if e == E and page % E == 0 and vs == (*lead, page // E, U * E, E) and k_pages.dtype is dtype and v_pages.dtype is dtype \
                and k_pages.get_device() == dev and v_pages.get_device() == dev and k_pages.is_contiguous() and v_pages.is_contiguous():
            return lead[-2], lead[-1], U * E, page
    if len(ks) != dims or len(vs) != dims:
        raise ValueError(f"k_pages and v_pages must have {dims} dimensions")
    if k_pages.dtype is not dtype or v_pages.dtype is not dtype:
        raise TypeError(f"k_pages and v_pages must be {dtype}, got {k_pages.dtype} and {v_pages.dtype}")
    if k_pages.get_device() != dev or v_pages.get_device() != dev:
        raise ValueError(f"k_pages and v_pages must be on device {dev}, got {k_pages.device} and {v_pages.device}")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    raise ValueError(f"k_pages must be [..., P, Hkv, D / {E}, page_size, {E}] and v_pages [..., P, Hkv, page_size / {E}, D, {E}], "
                     f"got {tuple(ks)} and {tuple(vs)}")


def _rows(t, name: str, shape: tuple, dtype, dev: int):
    """Address and strides (sequence, node) of a [B, N, H, D] tensor whose heads lie together."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        sb, sn, sh, sd = t.stride()
        B, N, H, D = shape
        if B | N | H > 0x7FFFFFFF:
            _too_large(name, B, N, H)
        if sd == 1 and sh == D or (sd == 1 or D <= 1) and (sh == D or H <= 1):
            # a dimension of one entry may carry any stride: it is never stepped
            return t.data_ptr(), sb if B > 1 else 0, sn if N > 1 else 0
        raise ValueError(f"{name}'s heads must lie together (strides D and 1), got strides {t.stride()}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be on device {dev}, got {t.device}")


def _table(t, dev: int, rows: int | None = None):
    """Address and width of a page table."""
    if t.dim() != 2:
        raise ValueError("page_table must have two dimensions, sequences and pages")
    B, W = t.shape
    if B | W > 0x7FFFFFFF:
        _too_large("page_table", B, W)
    return _ints(t, "page_table", (B if rows is None else rows, W), dev), W


def _device(t, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _elsewhere(dev: int, stream):
    """None if a call may allocate and launch as things are; else the context to do it in: the
    tensors' device current and, given a raw stream of the caller's, that stream current too, so
    that what the call allocates belongs to it."""
    if stream is not None:
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev))
    return None if dev == _current_device() else torch.cuda.device(dev)


def _work(workspace, nbytes: int, dev: int):
    if workspace is None:
        return torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=dev)
    if workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on device {dev}")
    return workspace


def _raise(rc: int):
    if rc != 0:
        raise SpecVerifyError(rc, sv_status_string(rc))


# Bounded: a server's batch sizes and table widths go on changing.
@lru_cache(maxsize=1024)
def _attention_bytes(*sizes) -> int:
    return int(load_library().sv_attention_workspace_bytes(*sizes))


@lru_cache(maxsize=1024)
def _resize_bytes(*sizes) -> int:
    return int(load_library().sv_resize_workspace_bytes(*sizes))


def sv_attention_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, D: int, page_size: int, table_width: int,
                                 dtype: int) -> int:
    return int(load_library().sv_attention_workspace_bytes(B, N, Hq, Hkv, D, page_size, table_width, dtype))


def sv_resize_workspace_bytes(S: int, num_pages: int) -> int:
    return int(load_library().sv_resize_workspace_bytes(S, num_pages))


def sv_attention_launch_plan(N: int, Hq: int, Hkv: int, D: int, dtype: int) -> list[str]:
    s = load_library().sv_attention_launch_plan(N, Hq, Hkv, D, dtype).decode()
    return s.split(";") if s else []


def spec_paged_attention(q, k_pages, v_pages, page_table, cache_len, *, parent=None, n_new=None, scale: float | None = None,
                         window: int = 0, sinks: int = 0, prior=None, workspace=None, stream=None, out=None, events=None):
    """Attention of the new tokens over a paged cache (see include/spec_cache.h).

    q [B, N, Hq, D] bfloat16 or float32 (heads together, any strides between sequences and
    nodes), one layer's k_pages [P, Hkv, D/E, page, E] and v_pages [P, Hkv, page/E, D, E],
    page_table [B, W], cache_len [B], n_new [B] (None: N each), parent [B, N] (None: a chain)
    and prior [B] (row codes of an earlier call: a sequence with one has it again and rows of
    NaN) int32.  scale defaults to 1 / sqrt(D).  Returns (out [B, N, Hq, D], row_status [B]);
    ``out`` may supply the two tensors.  ``events`` as for spec_verify: the number of kernels is
    then returned last.
    """
    dev = _device(q, "q")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return spec_paged_attention(q, k_pages, v_pages, page_table, cache_len, parent=parent, n_new=n_new, scale=scale,
                                        window=window, sinks=sinks, prior=prior, workspace=workspace, out=out, events=events)
    dt = _code(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B, N, Hq, D]")
    shape = q.shape
    B, N, Hq, D = shape
    P, Hkv, Dk, page = _pages(k_pages, v_pages, 5, q.dtype, dev)
    if Dk != D:
        raise ValueError(f"the cache's heads have {Dk} elements, q's {D}")
    qp, qb, qn = _rows(q, "q", shape, q.dtype, dev)
    table, W = _table(page_table, dev, B)
    seqs = (B,)
    lens, news = _ints(cache_len, "cache_len", seqs, dev), _ints(n_new, "n_new", seqs, dev, True)
    par, pri = _ints(parent, "parent", (B, N), dev, True), _ints(prior, "prior", seqs, dev, True)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if window or sinks:
        _int32(window, "window"), _int32(sinks, "sinks")
    if out is not None:
        if not out[0].is_contiguous():
            raise ValueError("out must be contiguous")
        _rows(out[0], "out", shape, q.dtype, dev)
        _ints(out[1], "row_status", seqs, dev)
        _apart({"row_status": out[1]}, {"prior": prior})

    o, st = out or (torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(cache_len))
    ws = _work(workspace, _attention_bytes(B, N, Hq, Hkv, D, page, W, dt), dev)
    args = (qp, qb, qn, k_pages.data_ptr(), v_pages.data_ptr(), dt, table, lens, news, par, pri, B, N, Hq, Hkv, D, page, P, W,
            scale, window, sinks, o.data_ptr(), st.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if events is None:
        rc = load_library().spec_paged_attention_after(*args, None, 0, None)
        if rc:
            _raise(rc)
        return o, st
    n = ctypes.c_int32(0)
    _raise(load_library().spec_paged_attention_after(*args, (ctypes.c_void_p * len(events))(*events), len(events), ctypes.byref(n)))
    return o, st, n.value


def spec_cache_append(k, v, k_pages, v_pages, page_table, cache_len, *, n_new=None, prior=None, stream=None, out=None):
    """Writes the new tokens' keys and values k, v [B, N, Hkv, D] (heads together, any strides
    between sequences and nodes) into slots cache_len .. cache_len + n_new - 1 of one layer's
    k_pages and v_pages (see include/spec_cache.h); nothing for a sequence with a row code of an
    earlier call in prior [B] int32.  Returns row_status [B] int32, which ``out`` may supply."""
    dev = _device(k, "k")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return spec_cache_append(k, v, k_pages, v_pages, page_table, cache_len, n_new=n_new, prior=prior, out=out)
    dt = _code(k, "k")
    if k.dim() != 4:
        raise ValueError("k must be [B, N, Hkv, D]")
    shape = k.shape
    B, N, Hkv, D = shape
    P, Hc, Dk, page = _pages(k_pages, v_pages, 5, k.dtype, dev)
    if Hc != Hkv or Dk != D:
        raise ValueError(f"the cache has {Hc} heads of {Dk} elements, k {Hkv} of {D}")
    kp, kb, kn = _rows(k, "k", shape, k.dtype, dev)
    vp, vb, vn = _rows(v, "v", shape, k.dtype, dev)
    table, W = _table(page_table, dev, B)
    seqs = (B,)
    lens, news = _ints(cache_len, "cache_len", seqs, dev), _ints(n_new, "n_new", seqs, dev, True)
    pri = _ints(prior, "prior", seqs, dev, True)
    if out is not None:
        _ints(out, "row_status", seqs, dev)
        _apart({"row_status": out}, {"prior": prior})

    st = torch.empty_like(cache_len) if out is None else out
    rc = load_library().spec_cache_append_after(kp, kb, kn, vp, vb, vn, dt, k_pages.data_ptr(), v_pages.data_ptr(), table, lens,
                                                news, pri, B, N, Hkv, D, page, P, W, st.data_ptr(), _raw_stream(dev))
    if rc:
        _raise(rc)
    return st


def spec_cache_commit(k_pages, v_pages, page_table, cache_len, accepted_len, path_nodes=None, *, max_new: int | None = None,
                      prior=None, stream=None, out=None):
    """Keeps node 0 and the accepted nodes of every sequence in all layers of k_pages
    [L, P, Hkv, D/E, page, E] and v_pages (see include/spec_cache.h): accepted_len [B] and
    path_nodes [B, N] int32 as spec_tree_verify returns them, or for chains accepted_len alone
    and ``max_new``, the N = G + 1 new tokens that were verified.  A sequence with a row code of
    an earlier call in prior [B] int32 keeps its length and its entries.  Returns (new_len [B],
    row_status [B]) int32; ``out`` may supply them (for chains new_len may be cache_len itself)."""
    dev = _device(k_pages, "k_pages")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return spec_cache_commit(k_pages, v_pages, page_table, cache_len, accepted_len, path_nodes, max_new=max_new, prior=prior, out=out)
    dt = _code(k_pages, "k_pages")
    P, Hkv, D, page = _pages(k_pages, v_pages, 6, k_pages.dtype, dev)
    table, W = _table(page_table, dev)
    B = page_table.shape[0]
    if path_nodes is not None:
        N = _int32(path_nodes.shape[1], "path_nodes' nodes") if path_nodes.dim() == 2 else 0
        if max_new is not None and max_new != N:
            raise ValueError(f"path_nodes has {N} nodes, max_new is {max_new}")
    elif max_new is None:
        raise ValueError("chains need max_new, the new tokens N = G + 1 of the verification")
    else:
        N = _int32(max_new, "max_new")
    seqs = (B,)
    lens, acc = _ints(cache_len, "cache_len", seqs, dev), _ints(accepted_len, "accepted_len", seqs, dev)
    path, pri = _ints(path_nodes, "path_nodes", (B, N), dev, True), _ints(prior, "prior", seqs, dev, True)
    if out is not None:
        _ints(out[0], "new_len", seqs, dev)
        _ints(out[1], "row_status", seqs, dev)
        _apart({"new_len": out[0], "row_status": out[1]},
               {"prior": prior, **({"cache_len": cache_len, "accepted_len": accepted_len} if path_nodes is not None else {})})

    n, st = out or (torch.empty_like(cache_len), torch.empty_like(cache_len))
    rc = load_library().spec_cache_commit_after(k_pages.data_ptr(), v_pages.data_ptr(), dt, table, lens, acc, path, pri,
                                                k_pages.shape[0], B, N, Hkv, D, page, P, W, n.data_ptr(), st.data_ptr(),
                                                _raw_stream(dev))
    if rc:
        _raise(rc)
    return n, st


def _books(pool: PagePool, dev: int):
    table, W = _table(pool.page_table, dev)
    S, P = pool.page_table.shape[0], _int32(pool.ref_count.numel(), "the pool's pages")
    return S, W, P, (table, _ints(pool.seq_pages, "seq_pages", (S,), dev), _ints(pool.ref_count, "ref_count", (P,), dev))


def spec_cache_resize(pool: PagePool, keep_len, want_len, k_pages=None, v_pages=None, *, page_size: int | None = None,
                      workspace=None, stream=None, out=None):
    """Gives every sequence of the pool the pages for want_len [S] slots and takes back those
    behind (see include/spec_cache.h); a page that others hold too and that lies at or behind slot
    keep_len [S] is replaced by the sequence's own, its kept slots copied in all layers of k_pages
    [L, P, Hkv, D/E, page, E] and v_pages.  Without them nothing is copied and ``page_size`` is
    needed.  Returns row_status [S] int32, which ``out`` may supply; the calls that go on with the
    same sequences take it as ``prior``."""
    dev = _device(pool.page_table, "page_table")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return spec_cache_resize(pool, keep_len, want_len, k_pages, v_pages, page_size=page_size, workspace=workspace, out=out)
    S, W, P, books = _books(pool, dev)
    free = _ints(pool.free_map, "free_map", ((P + 31) // 32,), dev)
    if k_pages is not None:
        dt = _code(k_pages, "k_pages")
        Pc, Hkv, D, page = _pages(k_pages, v_pages, 6, k_pages.dtype, dev)
        if Pc != P:
            raise ValueError(f"the cache has {Pc} pages, the pool {P}")
        if page_size is not None and page_size != page:
            raise ValueError(f"the cache's pages have {page} slots, page_size is {page_size}")
        L, kp, vp = k_pages.shape[0], k_pages.data_ptr(), v_pages.data_ptr()
    elif page_size is None:
        raise ValueError("page_size is needed without k_pages and v_pages")
    else:
        dt, L, Hkv, D, page, kp, vp = SV_BF16, 0, 1, 16, _int32(page_size, "page_size"), None, None
    seqs = (S,)
    keep, want = _ints(keep_len, "keep_len", seqs, dev), _ints(want_len, "want_len", seqs, dev)
    if out is not None:
        _ints(out, "row_status", seqs, dev)

    st = torch.empty_like(keep_len) if out is None else out
    ws = _work(workspace, _resize_bytes(S, P), dev)
    rc = load_library().spec_cache_resize(*books, free, keep, want, kp, vp, dt, L, S, Hkv, D, page, P, W, st.data_ptr(),
                                          ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if rc:
        _raise(rc)
    return st


def spec_cache_fork(pool: PagePool, cache_len, src, dst, *, stream=None, out=None):
    """Makes sequences dst [F] continuations of sequences src [F] (int32) that share their pages
    (see include/spec_cache.h); cache_len [S] is written at dst.  Returns pair_status [F] int32,
    which ``out`` may supply."""
    dev = _device(pool.page_table, "page_table")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return spec_cache_fork(pool, cache_len, src, dst, out=out)
    S, W, P, books = _books(pool, dev)
    F = _int32(src.numel(), "the pairs")
    pairs = (F,)
    lens = _ints(cache_len, "cache_len", (S,), dev)
    s, d = _ints(src, "src", pairs, dev), _ints(dst, "dst", pairs, dev)
    if out is not None:
        _ints(out, "pair_status", pairs, dev)

    st = torch.empty_like(src) if out is None else out
    rc = load_library().spec_cache_fork(*books, lens, s, d, F, S, P, W, st.data_ptr(), _raw_stream(dev))
    if rc:
        _raise(rc)
    return st
