"""The paged cache: rows of any length on one pool of pages (see include/kvp.h).

A row is one (sequence or layer, KV head), as in the dense caches; its tokens live in pages that a
row of ``table`` names.  :class:`PagedCache` wraps the buffers and the functions beside it are the
C ABI's calls on them, with the checks of shapes, types and devices that need no look at the data.
What only the device can see (a length or page out of range, no free page left) is raised by
:func:`kvp_check_device_status`.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import _DTYPE, _check, _dtype, _need, load

# a call costs the host a few microseconds; making a Stream object would be a third of them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Desc(ctypes.Structure):
    """kvp_paged_cache."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pool", "v_pool")] + \
               [(n, ctypes.c_int64) for n in ("page_stride", "token_stride")] + \
               [(n, ctypes.c_void_p) for n in ("table", "lens", "refs", "free_mask", "score", "pos")] + \
               [(n, ctypes.c_int) for n in ("dtype", "head_dim", "page_size", "n_pages", "n_rows", "max_pages")]


class PagedCache:
    """The buffers of a paged cache, checked once.

    k_pool, v_pool [n_pages, page_size, head_dim] (views with a contiguous last axis and equal, non-zero
    strides will do: ``kv[:, 0]`` and ``kv[:, 1]`` of one [n_pages, 2, page_size, head_dim] buffer);
    table int32 [n_rows, max_pages]; lens int32 [n_rows]; refs int32 [n_pages]; free_mask int32
    [ceil(n_pages / 32)]; score float32 and pos int32 [n_rows, max_pages * page_size], each optional.
    The buffers hold a cache's books already, or :func:`kvp_paged_init` empties them;
    :meth:`empty` allocates a new cache.
    """

    def __init__(self, k_pool, v_pool, table, lens, refs, free_mask, score=None, pos=None):
        for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if not t.is_cuda or t.dim() != 3:
                raise ValueError(f"{name} must be a CUDA tensor [n_pages, page_size, head_dim]")
            if t.stride(2) != 1:
                raise ValueError(f"{name}: the head_dim axis must be contiguous")
            # 0 stands for the dense stride in the descriptor, so a broadcast axis would run past the pool
            if (t.shape[0] > 1 and t.stride(0) == 0) or (t.shape[1] > 1 and t.stride(1) == 0):
                raise ValueError(f"{name}: the page and token axes must not be broadcast")
        if v_pool.shape != k_pool.shape or v_pool.dtype != k_pool.dtype or v_pool.stride() != k_pool.stride():
            raise ValueError("k_pool and v_pool must have the same shape, dtype and strides")
        n_pages, page_size, head_dim = k_pool.shape
        _need(table, "table", torch.int32)
        if table.dim() != 2:
            raise ValueError("table must be [n_rows, max_pages]")
        n_rows, max_pages = table.shape
        _need(lens, "lens", torch.int32, (n_rows,))
        _need(refs, "refs", torch.int32, (n_pages,))
        _need(free_mask, "free_mask", torch.int32, ((n_pages + 31) // 32,))
        if score is not None:
            _need(score, "score", torch.float32, (n_rows, max_pages * page_size))
        if pos is not None:
            _need(pos, "pos", torch.int32, (n_rows, max_pages * page_size))
        self.device = k_pool.device
        for name, t in (("v_pool", v_pool), ("table", table), ("lens", lens), ("refs", refs),
                        ("free_mask", free_mask), ("score", score), ("pos", pos)):
            if t is not None and t.device != self.device:
                raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        self.k_pool, self.v_pool, self.table, self.lens = k_pool, v_pool, table, lens
        self.refs, self.free_mask, self.score, self.pos = refs, free_mask, score, pos
        self.dtype, self.n_rows, self.max_pages = k_pool.dtype, n_rows, max_pages
        self.n_pages, self.page_size, self.head_dim = n_pages, page_size, head_dim
        # strides of one-page (one-token) pools say nothing: 0 takes the dense ones
        self._desc = _Desc(k_pool.data_ptr(), v_pool.data_ptr(),
                           k_pool.stride(0) if n_pages > 1 else 0, k_pool.stride(1) if page_size > 1 else 0,
                           table.data_ptr(), lens.data_ptr(), refs.data_ptr(), free_mask.data_ptr(),
                           None if score is None else score.data_ptr(), None if pos is None else pos.data_ptr(),
                           _dtype(k_pool), head_dim, page_size, n_pages, n_rows, max_pages)
        self._ref = ctypes.byref(self._desc)
        self._index = self.device.index
        self._sizes = {}

    @classmethod
    def empty(cls, n_rows, max_pages, n_pages, page_size, head_dim, dtype=torch.bfloat16, device="cuda",
              scores=False, positions=False):
        """A new, empty cache; ``scores`` / ``positions``: with the per-slot arrays."""
        def make(*shape, dtype=torch.int32):
            return torch.empty(*shape, dtype=dtype, device=device)
        cap = max_pages * page_size
        c = cls(make(n_pages, page_size, head_dim, dtype=dtype), make(n_pages, page_size, head_dim, dtype=dtype),
                make(n_rows, max_pages), make(n_rows), make(n_pages), make((n_pages + 31) // 32),
                make(n_rows, cap, dtype=torch.float32).zero_() if scores else None,
                make(n_rows, cap).zero_() if positions else None)
        kvp_paged_init(c)
        return c

    def rows(self, start, stop):
        """The rows [start, stop) (one layer's, say) as a cache on the same pages and books."""
        if not 0 <= start < stop <= self.n_rows:
            raise ValueError(f"rows [{start}, {stop}) of {self.n_rows}")
        cut = (lambda t: None if t is None else t[start:stop])
        return PagedCache(self.k_pool, self.v_pool, self.table[start:stop], self.lens[start:stop], self.refs,
                          self.free_mask, cut(self.score), cut(self.pos))

    def _workspace(self, fn, *args):
        """A workspace for one call (from the caching allocator: calls that overlap have their own):
        (tensor, pointer, bytes)."""
        key = (fn, args)
        n = self._sizes.get(key)
        if n is None:
            n = self._sizes[key] = int(getattr(load(), fn + "_workspace_size")(self._ref, *args))
        if n == 0:
            return None, None, 0
        ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        return ws, ws.data_ptr(), n

    def _need(self, t, name, dtype, shape):
        _need(t, name, dtype, shape)
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")

    def _elsewhere(self, stream):
        """Whether the call has to be made under another device or stream than the current ones."""
        return stream is not None or torch.cuda.current_device() != self._index

    def _there(self, stream):
        """Makes them current, so that the call's temporaries belong to the stream that uses them."""
        if stream is None:
            return torch.cuda.device(self.device)
        if stream.device != self.device:
            raise ValueError(f"stream must be on {self.device}, got {stream.device}")
        return torch.cuda.stream(stream)


def _cache(c):
    if not isinstance(c, PagedCache):
        raise TypeError("cache must be a PagedCache")
    return c


def kvp_paged_init(cache, stream=None):
    """Empty the cache: no row holds a page."""
    if _cache(cache)._elsewhere(stream):
        with cache._there(stream):
            return kvp_paged_init(cache)
    _check("kvp_paged_init", load().kvp_paged_init(cache._ref, _raw_stream(cache._index)))


def _new_tokens(cache, t, name, like=None):
    """[R, n_new, D] or [B, h_kv, n_new, D] with a contiguous last axis: (h_kv, n_new, strides or None)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device}, got {t.device}")
    if t.dtype != cache.dtype:
        raise ValueError(f"{name} must be {cache.dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) == 3 and shape[0] == cache.n_rows and shape[2] == cache.head_dim:
        h_kv, n_new = shape[0], shape[1]
    elif len(shape) == 4 and shape[0] * shape[1] == cache.n_rows and shape[3] == cache.head_dim:
        h_kv, n_new = shape[1], shape[2]
    else:
        raise ValueError(f"{name} must be [{cache.n_rows}, n_new, {cache.head_dim}] or [batch, h_kv, n_new, "
                         f"{cache.head_dim}] with batch * h_kv = {cache.n_rows}, got {tuple(shape)}")
    if like is not None and shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(shape)}")
    if t.is_contiguous():
        return h_kv, n_new, None
    strides = t.stride()
    if strides[-1] != 1:
        raise ValueError(f"{name}: the head_dim axis must be contiguous")
    return h_kv, n_new, (ctypes.c_int64 * 3)(strides[0] if len(shape) == 4 else 0, strides[-3], strides[-2])


def kvp_paged_append(cache, new_k, new_v, counts=None, new_pos=None, stream=None):
    """Append ``counts`` (int32 [R]; None: all) of the new tokens to every row: new_k, new_v
    [R, n_new, D] or [batch, h_kv, n_new, D] (strided views are read in place).  new_pos int32 [R]:
    the source position of each row's first new token, for a cache with ``pos``."""
    if _cache(cache)._elsewhere(stream):
        with cache._there(stream):
            return kvp_paged_append(cache, new_k, new_v, counts, new_pos)
    h_kv, n_new, ks = _new_tokens(cache, new_k, "new_k")
    vs = _new_tokens(cache, new_v, "new_v", new_k)[2]
    if counts is not None:
        cache._need(counts, "counts", torch.int32, (cache.n_rows,))
    if new_pos is not None:
        cache._need(new_pos, "new_pos", torch.int32, (cache.n_rows,))
    ws, ws_ptr, ws_bytes = cache._workspace("kvp_paged_append", n_new)
    rc = load().kvp_paged_append(cache._ref, new_k.data_ptr(), new_v.data_ptr(), ks, vs, h_kv, n_new,
                                 None if counts is None else counts.data_ptr(),
                                 None if new_pos is None else new_pos.data_ptr(), ws_ptr, ws_bytes,
                                 _raw_stream(cache._index))
    _check("kvp_paged_append", rc)


def kvp_paged_fork(cache, src, copy=False, stream=None):
    """Give every row r with src[r] >= 0 (int32 [R]) the tokens of row src[r]: on the same pages, or
    (copy) on fresh ones."""
    if _cache(cache)._elsewhere(stream):
        with cache._there(stream):
            return kvp_paged_fork(cache, src, copy)
    cache._need(src, "src", torch.int32, (cache.n_rows,))
    copy = int(bool(copy))
    ws, ws_ptr, ws_bytes = cache._workspace("kvp_paged_fork", copy)
    _check("kvp_paged_fork", load().kvp_paged_fork(cache._ref, src.data_ptr(), copy, ws_ptr, ws_bytes,
                                                   _raw_stream(cache._index)))


def kvp_paged_compact(cache, idx, count, stream=None):
    """Keep, in place, the tokens idx [R, b_max] (int32, ascending) of every row, count [R] of them
    (negative: leave the row), and release the pages that empties.  A row whose indices are not all its
    own, or do not ascend, stays as it is and raises the device status.

    kvp_select_topk takes one length for all rows.  For rows of different lengths give it scores that are
    NaN (ranked last) behind each row's end and +inf where a token is to be kept in any case::

        col, n = torch.arange(T, device=cache.device), cache.lens[:, None]
        score = torch.where((col < n_sink) | (col >= n - n_recent), math.inf, cache.score[:, :T])
        score = torch.where(col < n, score, math.nan)
        idx, count = kvp_select_topk(score, torch.minimum(budgets, cache.lens), 0, 0, b_max, T=T)
    """
    if _cache(cache)._elsewhere(stream):
        with cache._there(stream):
            return kvp_paged_compact(cache, idx, count)
    cache._need(idx, "idx", torch.int32, None)
    if idx.dim() != 2 or idx.shape[0] != cache.n_rows:
        raise ValueError(f"idx must be [{cache.n_rows}, b_max], got {tuple(idx.shape)}")
    cache._need(count, "count", torch.int32, (cache.n_rows,))
    b_max = idx.shape[1]
    ws, ws_ptr, ws_bytes = cache._workspace("kvp_paged_compact", b_max)
    _check("kvp_paged_compact", load().kvp_paged_compact(cache._ref, idx.data_ptr(), count.data_ptr(), b_max, ws_ptr,
                                                         ws_bytes, _raw_stream(cache._index)))


def kvp_paged_free(cache, keep=None, stream=None):
    """Cut every row r to keep[r] tokens (int32 [R]; negative: leave the row; None: empty all rows)."""
    if _cache(cache)._elsewhere(stream):
        with cache._there(stream):
            return kvp_paged_free(cache, keep)
    if keep is not None:
        cache._need(keep, "keep", torch.int32, (cache.n_rows,))
    _check("kvp_paged_free", load().kvp_paged_free(cache._ref, None if keep is None else keep.data_ptr(),
                                                   _raw_stream(cache._index)))


def kvp_paged_decode_attn(q, cache, sm_scale=None, out=None, out_dtype=None, lse=None, return_lse=False,
                          add_scores=False, workspace=None, stream=None):
    """One-token attention over the paged rows: q [L, H_q, D] (the layer axis may be strided), rows
    r = l * h_kv + h -> out [L, H_q, D] float32 (or ``out_dtype`` = the cache's dtype); with
    ``return_lse`` (out, lse float32 [L, H_q]).  ``add_scores`` adds every token's probability,
    summed over its group, to ``cache.score``."""
    if _cache(cache)._elsewhere(stream):
        with cache._there(stream):
            return kvp_paged_decode_attn(q, cache, sm_scale, out, out_dtype, lse, return_lse, add_scores, workspace)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.device != cache.device:
        raise ValueError(f"q must be on {cache.device}, got {q.device}")
    D = cache.head_dim
    if q.dim() != 3 or q.dtype != cache.dtype or q.shape[2] != D:
        raise ValueError(f"q must be {cache.dtype} [n_layers, h_q, {D}], got {q.dtype} {tuple(q.shape)}")
    L, Hq, _ = q.shape
    if L < 1 or cache.n_rows % L:
        raise ValueError("the cache's rows must be n_layers * h_kv")
    q_stride = 0                                   # dense
    if not q.is_contiguous():
        if q.stride(2) != 1 or (q.stride(1) != D and Hq > 1):
            raise ValueError("q: the head and head_dim axes must be contiguous")
        if L > 1:
            q_stride = q.stride(0)
            if q_stride == 0:
                raise ValueError("q: the layer axis must not be broadcast")
    h_kv = cache.n_rows // L
    add_scores = int(bool(add_scores))
    if out is None:
        out = torch.empty((L, Hq, D), dtype=out_dtype or torch.float32, device=cache.device)
    else:
        cache._need(out, "out", out_dtype, (L, Hq, D))
    if out.dtype not in _DTYPE:
        raise ValueError(f"unsupported out dtype {out.dtype}")
    if lse is not None:
        cache._need(lse, "lse", torch.float32, (L, Hq))
    elif return_lse:
        lse = torch.empty((L, Hq), dtype=torch.float32, device=cache.device)
    if workspace is None:
        workspace, ws_ptr, ws_bytes = cache._workspace("kvp_paged_decode_attn", Hq, h_kv, add_scores)
    else:
        cache._need(workspace, "workspace", torch.uint8, None)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
    rc = load().kvp_paged_decode_attn(q.data_ptr(), q_stride, cache._ref, Hq, h_kv,
                                      D ** -0.5 if sm_scale is None else float(sm_scale), out.data_ptr(),
                                      _DTYPE[out.dtype], None if lse is None else lse.data_ptr(), add_scores, ws_ptr,
                                      ws_bytes, _raw_stream(cache._index))
    _check("kvp_paged_decode_attn", rc)
    return (out, lse) if return_lse else out
