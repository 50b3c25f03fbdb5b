"""Binding of the serving operators: the paged K/V cache, attention over it, page
management and token log-probabilities (include/dspark.h).

As in ``binding``: tensors are checked on the host, their pointers go to the
C-ABI with the current CUDA stream (or ``stream``), nothing synchronises and
there is no fallback.  Outputs and workspaces are allocated where the caller
gives none; a loop passes the returned ``workspace`` back in.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .binding import DSparkError, _dtype_code, load

DEV_NO_PAGES = 4

_I32, _F32 = torch.int32, torch.float32


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + \
        [(n, ctypes.c_int) for n in ("dtype", "layers", "n_pages", "page_size", "heads", "head_dim")] + \
        [(n, ctypes.c_longlong) for n in ("layer_stride", "page_stride", "token_stride", "head_stride")]


def _strides(t):
    """Strides, those of dimensions of one, which carry no meaning, as those of an array without gaps."""
    out, dense = [], 1
    for n, s in zip(reversed(t.shape), reversed(t.stride())):
        out.append(dense if n == 1 else s)
        dense = (dense if n == 1 else s) * n
    return out[::-1]


class PagedCache:
    """K and V of all layers as pages: ``k``, ``v`` [layers, n_pages, page_size, heads, head_dim]
    (float32 or bfloat16) with any strides, the same for both, and head_dim contiguous.  A pool
    stored heads-first is passed as ``pool.transpose(2, 3)``.  Keeps references, copies nothing."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a CUDA tensor")
            if t.dim() != 5:
                raise ValueError(f"{name} must be [layers, n_pages, page_size, heads, head_dim], got {tuple(t.shape)}")
            if t.stride(4) != 1 and t.shape[4] > 1:
                raise ValueError(f"{name}: head_dim must be contiguous")
        if k.shape != v.shape or k.dtype != v.dtype or _strides(k) != _strides(v) or k.device != v.device:
            raise ValueError("k and v must agree in shape, dtype, strides and device")
        self.k, self.v = k, v
        self.layers, self.n_pages, self.page_size, self.heads, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), _dtype_code(k), *k.shape, *_strides(k)[:4])
        self.ref = ctypes.byref(self.struct)
        self.attention_bytes = None  # workspace of dspark_paged_attention, once asked for


def _dev(t, name, dtype, shape, dev):
    """Pointer of a contiguous tensor of this dtype, shape (None: any) and device."""
    try:
        if t.dtype is dtype and t.device == dev and t.is_contiguous() and (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _count(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.numel()


def _cache(cache):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    return cache


def _rows(t, name, dtype, heads, dim, dev):
    """Pointer and (token, head) strides of [n, heads, dim] rows whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim}], got {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    ts, hs, ds = st
    if ds != 1 and dim > 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    n, h, _ = shape
    if h == 1:  # the stride of a dimension of one carries no meaning
        hs = dim
    if n <= 1:
        ts = h * hs
    return t.data_ptr(), ts, hs


def _stream(dev, stream) -> int:
    """Handle of the launch stream: the device's current one, or the one given.  The device has to be
    the current one, where launches go."""
    if torch._C._cuda_getDevice() != dev.index:
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _new(shape, dtype, dev, stream):
    """A tensor for the launch stream: of that stream's memory, since a block of the current stream's
    may still be in use there by work launched before it was freed.  The current stream, where the
    caller mostly reads it, is recorded as a user."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    current = torch.cuda.current_stream(dev)
    if current != stream:
        t.record_stream(current)
    return t


def _out(t, name, shape, dtype, dev, stream):
    """The output tensor given, checked, or a new one; and its pointer."""
    if t is None:
        t = _new(shape, dtype, dev, stream)
        return t, t.data_ptr()
    return t, _dev(t, name, dtype, shape, dev)


def _workspace(nbytes, ws, dev, stream):
    """The workspace, its pointer and its size in bytes."""
    if ws is None:
        ws = _new((nbytes if nbytes > 256 else 256,), torch.uint8, dev, stream)
    elif ws.device != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < nbytes:
        raise ValueError(f"workspace needs {nbytes} contiguous bytes on {dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


@functools.lru_cache(maxsize=256)
def pages_workspace_bytes(R: int, n_pages: int) -> int:
    return int(load().dspark_pages_workspace_bytes(R, n_pages))


@functools.lru_cache(maxsize=256)
def logprobs_workspace_bytes(n_rows: int, V: int) -> int:
    return int(load().dspark_logprobs_workspace_bytes(n_rows, V))


def paged_attention_workspace_bytes(cache: PagedCache) -> int:
    if cache.attention_bytes is None:
        cache.attention_bytes = int(load().dspark_paged_attention_workspace_bytes(cache.ref))
    return cache.attention_bytes


def _table(page_table, dev):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [R, max_pages]")
    R, P = page_table.shape
    return R, P, _dev(page_table, "page_table", _I32, None, dev)


def dspark_cache_append(cache: PagedCache, layer: int, k_new, v_new, q_offsets, kv_len, page_table, *,
                        workspace=None, stream=None) -> dict:
    """Write the chunk's K and V (k_new, v_new [tokens, heads, head_dim], the same strides) of one
    layer.  q_offsets [R + 1], kv_len [R] (new tokens included), page_table [R, max_pages]: int32."""
    dev = _cache(cache).device
    kp, ts, hs = _rows(k_new, "k_new", cache.dtype, cache.heads, cache.head_dim, dev)
    vp, vts, vhs = _rows(v_new, "v_new", cache.dtype, cache.heads, cache.head_dim, dev)
    T = k_new.shape[0]
    if v_new.shape[0] != T or ts != vts or hs != vhs:
        raise ValueError("k_new and v_new must agree in shape and strides")
    R, P, pt = _table(page_table, dev)
    off = _dev(q_offsets, "q_offsets", _I32, (R + 1,), dev)
    kl = _dev(kv_len, "kv_len", _I32, (R,), dev)
    ws, wp, wn = _workspace(256, workspace, dev, stream)
    st = load().dspark_cache_append(cache.ref, layer, kp, vp, ts, hs, off, kl, pt, R, T, P, wp, wn,
                                    _stream(dev, stream))
    if st:
        raise DSparkError("dspark_cache_append", st)
    return dict(workspace=ws)


def dspark_paged_attention(q, cache: PagedCache, layer: int, q_offsets, kv_len, page_table, scale: float, *,
                           out=None, lse=None, workspace=None, stream=None) -> dict:
    """Attention of the chunk over one layer.  q [tokens, Hq, head_dim] (strided); returns
    out [tokens, Hq, head_dim] in the cache's dtype and lse [tokens, Hq] float32."""
    dev = _cache(cache).device
    qp, ts, hs = _rows(q, "q", cache.dtype, None, cache.head_dim, dev)
    T, Hq, D = q.shape
    R, P, pt = _table(page_table, dev)
    off = _dev(q_offsets, "q_offsets", _I32, (R + 1,), dev)
    kl = _dev(kv_len, "kv_len", _I32, (R,), dev)
    out, op = _out(out, "out", (T, Hq, D), cache.dtype, dev, stream)
    lse, lp = _out(lse, "lse", (T, Hq), _F32, dev, stream)
    ws, wp, wn = _workspace(paged_attention_workspace_bytes(cache), workspace, dev, stream)
    st = load().dspark_paged_attention(qp, ts, hs, Hq, cache.ref, layer, off, kl, pt, R, T, P, scale, op, lp, wp,
                                       wn, _stream(dev, stream))
    if st:
        raise DSparkError("dspark_paged_attention", st)
    return dict(out=out, lse=lse, workspace=ws)


def _meta(cache, page_table, kv_len, refcount, dev):
    R, P, pt = _table(page_table, dev)
    return R, P, pt, _dev(kv_len, "kv_len", _I32, (R,), dev), _dev(refcount, "refcount", _I32, (cache.n_pages,), dev)


def dspark_pages_resize(cache: PagedCache, page_table, kv_len, new_len, refcount, *, page_table_out=None,
                        kv_len_out=None, refcount_out=None, free_pages=None, workspace=None, stream=None) -> dict:
    """Give every request room for new_len positions: pages past it are freed, missing ones taken.
    The outputs may be the inputs' own tensors (in place)."""
    dev, n = _cache(cache).device, cache.n_pages
    R, P, pt, kl, rc = _meta(cache, page_table, kv_len, refcount, dev)
    nl = _dev(new_len, "new_len", _I32, (R,), dev)
    pto, ptp = _out(page_table_out, "page_table_out", (R, P), _I32, dev, stream)
    klo, klp = _out(kv_len_out, "kv_len_out", (R,), _I32, dev, stream)
    rco, rcp = _out(refcount_out, "refcount_out", (n,), _I32, dev, stream)
    fp, fpp = _out(free_pages, "free_pages", (1,), _I32, dev, stream)
    ws, wp, wn = _workspace(pages_workspace_bytes(R, n), workspace, dev, stream)
    st = load().dspark_pages_resize(cache.ref, pt, kl, nl, rc, R, P, ptp, klp, rcp, fpp, wp, wn,
                                    _stream(dev, stream))
    if st:
        raise DSparkError("dspark_pages_resize", st)
    return dict(page_table=pto, kv_len=klo, refcount=rco, free_pages=fp, workspace=ws)


def dspark_pages_fork(cache: PagedCache, page_table, kv_len, parent, child, refcount, *, page_table_out=None,
                      kv_len_out=None, refcount_out=None, free_pages=None, workspace=None, stream=None) -> dict:
    """Requests child[i] become copies of parent[i] (int32 [n]): full pages shared, the last one copied."""
    dev, n_pages = _cache(cache).device, cache.n_pages
    R, P, pt, kl, rc = _meta(cache, page_table, kv_len, refcount, dev)
    n = _count(parent, "parent")
    pa = _dev(parent, "parent", _I32, (n,), dev)
    ch = _dev(child, "child", _I32, (n,), dev)
    pto, ptp = _out(page_table_out, "page_table_out", (R, P), _I32, dev, stream)
    klo, klp = _out(kv_len_out, "kv_len_out", (R,), _I32, dev, stream)
    rco, rcp = _out(refcount_out, "refcount_out", (n_pages,), _I32, dev, stream)
    fp, fpp = _out(free_pages, "free_pages", (1,), _I32, dev, stream)
    ws, wp, wn = _workspace(pages_workspace_bytes(R, n_pages), workspace, dev, stream)
    st = load().dspark_pages_fork(cache.ref, pt, kl, rc, pa, ch, n, R, P, ptp, klp, rcp, fpp, wp, wn,
                                  _stream(dev, stream))
    if st:
        raise DSparkError("dspark_pages_fork", st)
    return dict(page_table=pto, kv_len=klo, refcount=rco, free_pages=fp, workspace=ws)


def dspark_pages_compact(cache: PagedCache, page_table, kv_len, refcount, *, page_table_out=None,
                         refcount_out=None, page_map=None, n_live=None, workspace=None, stream=None) -> dict:
    """Move the live pages to the lowest ids; page_map[p] is page p's id afterwards (-1: free)."""
    dev, n = _cache(cache).device, cache.n_pages
    R, P, pt, kl, rc = _meta(cache, page_table, kv_len, refcount, dev)
    pto, ptp = _out(page_table_out, "page_table_out", (R, P), _I32, dev, stream)
    rco, rcp = _out(refcount_out, "refcount_out", (n,), _I32, dev, stream)
    pm, pmp = _out(page_map, "page_map", (n,), _I32, dev, stream)
    nl, nlp = _out(n_live, "n_live", (1,), _I32, dev, stream)
    ws, wp, wn = _workspace(pages_workspace_bytes(R, n), workspace, dev, stream)
    st = load().dspark_pages_compact(cache.ref, pt, kl, rc, R, P, ptp, rcp, pmp, nlp, wp, wn, _stream(dev, stream))
    if st:
        raise DSparkError("dspark_pages_compact", st)
    return dict(page_table=pto, refcount=rco, page_map=pm, n_live=nl, workspace=ws)


def dspark_pages_copy(cache: PagedCache, src, dst, *, workspace=None, stream=None) -> dict:
    """Copy pages src[i] -> dst[i] (int32 [n]) of K and V in all layers."""
    dev = _cache(cache).device
    n = _count(src, "src")
    sp = _dev(src, "src", _I32, (n,), dev)
    dp = _dev(dst, "dst", _I32, (n,), dev)
    ws, wp, wn = _workspace(256, workspace, dev, stream)
    st = load().dspark_pages_copy(cache.ref, sp, dp, n, wp, wn, _stream(dev, stream))
    if st:
        raise DSparkError("dspark_pages_copy", st)
    return dict(workspace=ws)


def dspark_logprobs(Z, tokens, temperature: float = 1.0, top: int = 0, *, logp=None, entropy=None, lse=None,
                    top_ids=None, top_logp=None, workspace=None, stream=None) -> dict:
    """Log-probability of ``tokens`` [...] int32 under logits Z [..., V] (float32 or bfloat16), the
    distribution's entropy and log-sum-exp, and the ``top`` best ids with theirs.  Rows with a negative
    token are skipped (NaN, -1): Z and dspark_verify's ``tokens`` fit as they are.  Z's rows may be
    strided: all leading dimensions together have to step evenly."""
    if not isinstance(Z, torch.Tensor) or not Z.is_cuda:
        raise TypeError("Z must be a CUDA tensor")
    dev, lead, V = Z.device, Z.shape[:-1], Z.shape[-1]
    tk = _dev(tokens, "tokens", _I32, lead, dev)
    n = tokens.numel()
    if Z.stride(-1) != 1:
        raise ValueError("Z: the vocabulary must be contiguous")
    step = _row_step(Z)
    if step is None:
        raise ValueError("Z: the leading dimensions must step evenly")
    logp, p0 = _out(logp, "logp", lead, _F32, dev, stream)
    entropy, p1 = _out(entropy, "entropy", lead, _F32, dev, stream)
    lse, p2 = _out(lse, "lse", lead, _F32, dev, stream)
    top_ids, p3 = _out(top_ids, "top_ids", (*lead, top), _I32, dev, stream)
    top_logp, p4 = _out(top_logp, "top_logp", (*lead, top), _F32, dev, stream)
    ws, wp, wn = _workspace(logprobs_workspace_bytes(n, V), workspace, dev, stream)
    if not n:  # no rows: a clean status and nothing else
        with torch.cuda.stream(stream):
            ws.zero_()
    st = load().dspark_logprobs(Z.data_ptr(), _dtype_code(Z), step, tk, n, V, temperature, top, p0, p1, p2, p3, p4,
                                wp, wn, _stream(dev, stream)) if n else 0
    if st:
        raise DSparkError("dspark_logprobs", st)
    return dict(logp=logp, entropy=entropy, lse=lse, top_ids=top_ids, top_logp=top_logp, workspace=ws)


def _row_step(Z):
    """Elements from a row of Z (all but the last dimension) to the next; None: they do not step evenly."""
    if Z.is_contiguous():
        return Z.shape[-1]
    step = want = None
    for n, s in zip(Z.shape[-2::-1], Z.stride()[-2::-1]):
        if n == 1:  # its stride carries no meaning
            continue
        if step is None:
            step = s
        elif s != want:
            return None
        want = s * n
    return Z.shape[-1] if step is None else step
