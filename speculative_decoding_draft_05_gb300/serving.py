"""Binding of the serving operators: the paged K/V cache, attention over it, page
management and token log-probabilities (include/dspark.h).

As in ``binding``: tensors are checked on the host, their pointers go to the
C-ABI with the current CUDA stream (or ``stream``), nothing synchronises and
there is no fallback.  Outputs and workspaces are allocated where the caller
gives none; a loop passes the returned ``workspace`` back in.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import DSparkError, _check, _dtype_code, load  # noqa: F401

DEV_NO_PAGES = 4

_I32, _F32 = torch.int32, torch.float32


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + \
        [(n, ctypes.c_int) for n in ("dtype", "layers", "n_pages", "page_size", "heads", "head_dim")] + \
        [(n, ctypes.c_longlong) for n in ("layer_stride", "page_stride", "token_stride", "head_stride")]


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
        if k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must agree in shape, dtype, strides and device")
        self.k, self.v = k, v
        self.layers, self.n_pages, self.page_size, self.heads, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        # the stride of a dimension of size 1 carries no meaning; the library wants it positive
        st = [max(1, s) if n == 1 else s for s, n in zip(k.stride(), k.shape)]
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), _dtype_code(k), *k.shape, *st[:4])
        self.ref = ctypes.byref(self.struct)


def _dev(t, name, dtype=None, shape=None, dev=None):
    """Pointer of a contiguous device tensor of this dtype and shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return t.data_ptr()


def _cache(cache, dev=None):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    return cache


def _rows(t, name, dtype, heads, dim, dev):
    """Pointer and (token, head) strides of [n, heads, dim] rows whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or t.shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim}], got {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 and dim > 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return t.data_ptr(), st[0], st[1]


class _Alloc:
    """The launch stream of a call, and tensors that live on it."""

    def __init__(self, dev, stream):
        self.dev, self.given = dev, stream
        self.handle = (torch.cuda.current_stream(dev) if stream is None else stream).cuda_stream

    def new(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.dev)
        if self.given is not None:  # allocated on the current stream, used on another
            t.record_stream(self.given)
        return t

    def out(self, t, name, shape, dtype):
        if t is None:
            return self.new(shape, dtype)
        _dev(t, name, dtype, torch.Size(shape), self.dev)
        return t

    def workspace(self, nbytes, ws):
        if ws is None:
            return self.new((max(nbytes, 256),), torch.uint8)
        if ws.device != self.dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} contiguous bytes on {self.dev}")
        return ws


def _chunk(q_offsets, kv_len, page_table, dev):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [R, max_pages]")
    R, P = page_table.shape
    return (_dev(q_offsets, "q_offsets", _I32, torch.Size((R + 1,)), dev),
            _dev(kv_len, "kv_len", _I32, torch.Size((R,)), dev),
            _dev(page_table, "page_table", _I32, None, dev), R, P)


def dspark_cache_append(cache: PagedCache, layer: int, k_new, v_new, q_offsets, kv_len, page_table, *,
                        workspace=None, stream=None) -> dict:
    """Write the chunk's K and V (k_new, v_new [tokens, heads, head_dim], the same strides) of one
    layer.  q_offsets [R + 1], kv_len [R] (new tokens included), page_table [R, max_pages]: int32."""
    L = load()
    dev = _cache(cache).device
    a = _Alloc(dev, stream)
    kp, ts, hs = _rows(k_new, "k_new", cache.dtype, cache.heads, cache.head_dim, dev)
    vp, vts, vhs = _rows(v_new, "v_new", cache.dtype, cache.heads, cache.head_dim, dev)
    if k_new.shape != v_new.shape or (ts, hs) != (vts, vhs):
        raise ValueError("k_new and v_new must agree in shape and strides")
    off, kl, pt, R, P = _chunk(q_offsets, kv_len, page_table, dev)
    ws = a.workspace(256, workspace)
    if k_new.shape[0]:
        _check("dspark_cache_append", L.dspark_cache_append(
            cache.ref, layer, kp, vp, ts, hs, off, kl, pt, R, k_new.shape[0], P, ws.data_ptr(), ws.numel(), a.handle))
    return dict(workspace=ws)


def paged_attention_workspace_bytes(cache: PagedCache) -> int:
    return int(load().dspark_paged_attention_workspace_bytes(cache.ref))


def dspark_paged_attention(q, cache: PagedCache, layer: int, q_offsets, kv_len, page_table, scale: float, *,
                           out=None, lse=None, workspace=None, stream=None) -> dict:
    """Attention of the chunk over one layer.  q [tokens, Hq, head_dim] (strided); returns
    out [tokens, Hq, head_dim] in the cache's dtype and lse [tokens, Hq] float32."""
    L = load()
    dev = _cache(cache).device
    a = _Alloc(dev, stream)
    qp, ts, hs = _rows(q, "q", cache.dtype, None, cache.head_dim, dev)
    T, Hq, D = q.shape
    off, kl, pt, R, P = _chunk(q_offsets, kv_len, page_table, dev)
    out = a.out(out, "out", (T, Hq, D), cache.dtype)
    lse = a.out(lse, "lse", (T, Hq), _F32)
    ws = a.workspace(int(L.dspark_paged_attention_workspace_bytes(cache.ref)), workspace)
    if T:
        _check("dspark_paged_attention", L.dspark_paged_attention(
            qp, ts, hs, Hq, cache.ref, layer, off, kl, pt, R, T, P, scale, out.data_ptr(), lse.data_ptr(),
            ws.data_ptr(), ws.numel(), a.handle))
    return dict(out=out, lse=lse, workspace=ws)


def pages_workspace_bytes(R: int, n_pages: int) -> int:
    return int(load().dspark_pages_workspace_bytes(R, n_pages))


def _meta(cache, page_table, kv_len, refcount, dev):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [R, max_pages]")
    R, P = page_table.shape
    return (R, P, _dev(page_table, "page_table", _I32, None, dev),
            _dev(kv_len, "kv_len", _I32, torch.Size((R,)), dev),
            _dev(refcount, "refcount", _I32, torch.Size((cache.n_pages,)), dev))


def dspark_pages_resize(cache: PagedCache, page_table, kv_len, new_len, refcount, *, page_table_out=None,
                        kv_len_out=None, refcount_out=None, free_pages=None, workspace=None, stream=None) -> dict:
    """Give every request room for new_len positions: pages past it are freed, missing ones taken.
    The outputs may be the inputs' own tensors (in place)."""
    L = load()
    dev = _cache(cache).device
    a = _Alloc(dev, stream)
    R, P, pt, kl, rc = _meta(cache, page_table, kv_len, refcount, dev)
    nl = _dev(new_len, "new_len", _I32, torch.Size((R,)), dev)
    pto = a.out(page_table_out, "page_table_out", (R, P), _I32)
    klo = a.out(kv_len_out, "kv_len_out", (R,), _I32)
    rco = a.out(refcount_out, "refcount_out", (cache.n_pages,), _I32)
    fp = a.out(free_pages, "free_pages", (1,), _I32)
    ws = a.workspace(int(L.dspark_pages_workspace_bytes(R, cache.n_pages)), workspace)
    _check("dspark_pages_resize", L.dspark_pages_resize(
        cache.ref, pt, kl, nl, rc, R, P, pto.data_ptr(), klo.data_ptr(), rco.data_ptr(), fp.data_ptr(),
        ws.data_ptr(), ws.numel(), a.handle))
    return dict(page_table=pto, kv_len=klo, refcount=rco, free_pages=fp, workspace=ws)


def dspark_pages_fork(cache: PagedCache, page_table, kv_len, parent, child, refcount, *, page_table_out=None,
                      kv_len_out=None, refcount_out=None, free_pages=None, workspace=None, stream=None) -> dict:
    """Requests child[i] become copies of parent[i] (int32 [n]): full pages shared, the last one copied."""
    L = load()
    dev = _cache(cache).device
    a = _Alloc(dev, stream)
    R, P, pt, kl, rc = _meta(cache, page_table, kv_len, refcount, dev)
    n = parent.numel()
    pa = _dev(parent, "parent", _I32, torch.Size((n,)), dev)
    ch = _dev(child, "child", _I32, torch.Size((n,)), dev)
    pto = a.out(page_table_out, "page_table_out", (R, P), _I32)
    klo = a.out(kv_len_out, "kv_len_out", (R,), _I32)
    rco = a.out(refcount_out, "refcount_out", (cache.n_pages,), _I32)
    fp = a.out(free_pages, "free_pages", (1,), _I32)
    ws = a.workspace(int(L.dspark_pages_workspace_bytes(R, cache.n_pages)), workspace)
    _check("dspark_pages_fork", L.dspark_pages_fork(
        cache.ref, pt, kl, rc, pa, ch, n, R, P, pto.data_ptr(), klo.data_ptr(), rco.data_ptr(), fp.data_ptr(),
        ws.data_ptr(), ws.numel(), a.handle))
    return dict(page_table=pto, kv_len=klo, refcount=rco, free_pages=fp, workspace=ws)


def dspark_pages_compact(cache: PagedCache, page_table, kv_len, refcount, *, page_table_out=None,
                         refcount_out=None, page_map=None, n_live=None, workspace=None, stream=None) -> dict:
    """Move the live pages to the lowest ids; page_map[p] is page p's id afterwards (-1: free)."""
    L = load()
    dev = _cache(cache).device
    a = _Alloc(dev, stream)
    R, P, pt, kl, rc = _meta(cache, page_table, kv_len, refcount, dev)
    pto = a.out(page_table_out, "page_table_out", (R, P), _I32)
    rco = a.out(refcount_out, "refcount_out", (cache.n_pages,), _I32)
    pm = a.out(page_map, "page_map", (cache.n_pages,), _I32)
    nl = a.out(n_live, "n_live", (1,), _I32)
    ws = a.workspace(int(L.dspark_pages_workspace_bytes(R, cache.n_pages)), workspace)
    _check("dspark_pages_compact", L.dspark_pages_compact(
        cache.ref, pt, kl, rc, R, P, pto.data_ptr(), rco.data_ptr(), pm.data_ptr(), nl.data_ptr(),
        ws.data_ptr(), ws.numel(), a.handle))
    return dict(page_table=pto, refcount=rco, page_map=pm, n_live=nl, workspace=ws)


def dspark_pages_copy(cache: PagedCache, src, dst, *, workspace=None, stream=None) -> dict:
    """Copy pages src[i] -> dst[i] (int32 [n]) of K and V in all layers."""
    L = load()
    dev = _cache(cache).device
    a = _Alloc(dev, stream)
    n = src.numel()
    sp = _dev(src, "src", _I32, torch.Size((n,)), dev)
    dp = _dev(dst, "dst", _I32, torch.Size((n,)), dev)
    ws = a.workspace(256, workspace)
    if n:
        _check("dspark_pages_copy", L.dspark_pages_copy(cache.ref, sp, dp, n, ws.data_ptr(), ws.numel(), a.handle))
    return dict(workspace=ws)


def logprobs_workspace_bytes(n_rows: int, V: int) -> int:
    return int(load().dspark_logprobs_workspace_bytes(n_rows, V))


def dspark_logprobs(Z, tokens, temperature: float = 1.0, top: int = 0, *, logp=None, entropy=None, lse=None,
                    top_ids=None, top_logp=None, workspace=None, stream=None) -> dict:
    """Log-probability of ``tokens`` [...] int32 under logits Z [..., V] (float32 or bfloat16), the
    distribution's entropy and log-sum-exp, and the ``top`` best ids with theirs.  Rows with a negative
    token are skipped (NaN, -1): Z and dspark_verify's ``tokens`` fit as they are.  Z's rows may be
    strided: all leading dimensions together have to step evenly."""
    L = load()
    if not isinstance(Z, torch.Tensor) or not Z.is_cuda:
        raise TypeError("Z must be a CUDA tensor")
    dev, lead, V = Z.device, Z.shape[:-1], Z.shape[-1]
    a = _Alloc(dev, stream)
    tk = _dev(tokens, "tokens", _I32, lead, dev)
    n = tokens.numel()
    if Z.stride(-1) != 1:
        raise ValueError("Z: the vocabulary must be contiguous")
    if Z.dim() == 1:
        step = V
    elif Z.dim() == 2 or Z.is_contiguous():
        step = Z.stride(-2)
    else:
        step = Z.flatten(0, -2).stride(0) if _even(Z) else None
        if step is None:
            raise ValueError("Z: the leading dimensions must step evenly")
    if n == 1:
        step = V
    logp = a.out(logp, "logp", lead, _F32)
    entropy = a.out(entropy, "entropy", lead, _F32)
    lse = a.out(lse, "lse", lead, _F32)
    top_ids = a.out(top_ids, "top_ids", (*lead, top), _I32)
    top_logp = a.out(top_logp, "top_logp", (*lead, top), _F32)
    ws = a.workspace(int(L.dspark_logprobs_workspace_bytes(n, V)), workspace)
    if n:
        _check("dspark_logprobs", L.dspark_logprobs(
            Z.data_ptr(), _dtype_code(Z), step, tk, n, V, temperature, top, logp.data_ptr(), entropy.data_ptr(),
            lse.data_ptr(), top_ids.data_ptr(), top_logp.data_ptr(), ws.data_ptr(), ws.numel(), a.handle))
    return dict(logp=logp, entropy=entropy, lse=lse, top_ids=top_ids, top_logp=top_logp, workspace=ws)


def _even(Z) -> bool:
    """Whether Z's rows (all but the last dimension) lie one fixed step apart."""
    step = Z.stride(-2)
    for i in range(Z.dim() - 3, -1, -1):
        step *= Z.shape[i + 1]
        if Z.stride(i) != step:
            return False
    return True
