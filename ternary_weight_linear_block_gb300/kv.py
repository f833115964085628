"""The paged key/value cache and the verification of drafted-token trees.

What a decode step that verifies drafted tokens needs between its qkv and its
output linear, over the C entry points of the same names:

* ``kv_plan``: block tables and slot maps on the GPU from the requests' lengths;
* ``kv_write``: the new tokens' keys and values into the cache;
* ``tree_attention``: every row over its request's cached tokens and, of the
  request's new tokens, those that its mask names;
* ``kv_commit``: the accepted path of each tree made contiguous, all layers.

Lengths, tables, masks and paths are device tensors that only the kernels
read, so a step can be captured in a CUDA graph and replayed as they change.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Sequence

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.TERN_KV_BF16, torch.float16: B.TERN_KV_F16}


def _check(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _ints(t: torch.Tensor, name: str, dtype=torch.int32, ndim: int = 1):
    if not (t.is_cuda and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {ndim}-D CUDA tensor of {dtype}")


def _table(t: torch.Tensor, b: int):
    """Row stride and width of a block table (rows may be longer than the part in use)."""
    if t.is_cuda and t.dtype is torch.int32 and t.dim() == 2:
        rows, width = t.shape
        stride, one = t.stride()
        if rows == b and (one == 1 or width <= 1) and (stride >= width or b <= 1):
            return (stride if b > 1 else max(width, 1)), width
    raise ValueError("table: expected an int32 CUDA tensor [requests, width], rows dense")


def _heads(t: torch.Tensor, heads: int, dim: int, dtype, name: str):
    """Row and head strides of [rows, heads, dim], e.g. a slice of the qkv linear's output."""
    if t.is_cuda and t.dtype is dtype and t.dim() == 3:
        rows, h, d = t.shape
        row, head, one = t.stride()
        if h == heads and d == dim and one == 1:
            return (row if rows > 1 else heads * dim), (head if heads > 1 else dim)
    raise ValueError(f"{name}: expected a CUDA tensor [rows, {heads}, {dim}] of {dtype}, "
                     "dense along the last axis")


def _done(name: str, status: int):
    """The entry points are called without the wrappers of ``binding``: at decode
    sizes the wrappers would cost as much host time as the launch."""
    if status:
        raise B.TernError(name, status)


@functools.lru_cache(maxsize=None)
def _workspace_bytes(max_new: int, hq: int, heads: int, dim: int) -> int:
    return B.tern_tree_attention_workspace_bytes(max_new, hq, heads, dim)


def _on(stream):
    """Allocate on the stream that the call runs on."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


class KVCache:
    """Keys and values of one layer as pages: two tensors [pages, page_size,
    heads, dim] of bf16 or fp16 with the same strides (a permuted view of
    [pages, heads, page_size, dim] will do)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _check(k.is_cuda and k.ndim == 4 and k.dtype in _TYPES, "k: expected a 4-D CUDA tensor of bf16 or fp16")
        _check(v.is_cuda and v.device == k.device and v.dtype == k.dtype and v.shape == k.shape and
               v.stride() == k.stride(), "v: expected the device, type, shape and strides of k")
        _check(k.stride(3) == 1, "k, v: expected to be dense along the last axis")
        self.k, self.v = k, v
        self.pages, self.page_size, self.heads, self.dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        # an axis of length one may have any stride: give it one that passes
        ps, ts, hs = (k.stride(i) if k.shape[i] > 1 else self.page_size * self.heads * self.dim
                      for i in range(3))
        self.desc = B.KVCacheDesc(k.data_ptr(), v.data_ptr(), self.pages, self.page_size,
                                  self.heads, self.dim, ps, ts, hs, _TYPES[k.dtype])
        self.desc_bytes = bytes(self.desc)
        self.address = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int, dtype=torch.bfloat16,
              device="cuda", heads_first: bool = False) -> "KVCache":
        """A cache of uninitialised pages, rows of heads or (``heads_first``) heads of rows."""
        if heads_first:
            k, v = (torch.empty((pages, heads, page_size, dim), dtype=dtype, device=device)
                    .transpose(1, 2) for _ in range(2))
        else:
            k, v = (torch.empty((pages, page_size, heads, dim), dtype=dtype, device=device)
                    for _ in range(2))
        return cls(k, v)


class KVPlan(NamedTuple):
    row_start: torch.Tensor   # int32 [requests + 1]: first row of each request
    slots: torch.Tensor       # int64 [capacity]: where each row's keys and values go, -1: nowhere
    positions: torch.Tensor   # int32 [capacity]: each row's position in its request
    request: torch.Tensor     # int32 [capacity]: each row's request, -1 past the last
    info: torch.Tensor        # int32 [4]: rows, pages taken, next free_head, flags

    @classmethod
    def empty(cls, requests: int, capacity: int, device="cuda") -> "KVPlan":
        def ints(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=device)
        return cls(ints(requests + 1), ints(capacity, torch.int64), ints(capacity), ints(capacity),
                   ints(4))


def kv_plan(ctx_len: torch.Tensor, new_len: torch.Tensor, table: torch.Tensor,
            free_pages: torch.Tensor, page_size: int, capacity: int,
            free_head: torch.Tensor | None = None, plan: KVPlan | None = None,
            stream=None) -> KVPlan:
    """Block tables and slot maps of one step: request b gets new_len[b] rows
    behind its ctx_len[b] cached tokens; the pages that they need beyond
    those it has are taken from ``free_pages`` (from index free_head[0] on)
    and written into ``table`` in place.  ``capacity`` rows are planned;
    ``plan`` gives the outputs' buffers.  info[3] says what did not fit."""
    b = ctx_len.shape[0]
    _ints(ctx_len, "ctx_len")
    _ints(new_len, "new_len")
    _ints(free_pages, "free_pages")
    _check(new_len.shape[0] == b, "new_len: expected as many requests as ctx_len")
    stride, width = _table(table, b)
    if free_head is not None:
        _check(free_head.is_cuda and free_head.dtype == torch.int32 and free_head.numel() == 1,
               "free_head: expected one int32 on the GPU")
    if plan is None:
        if stream is None:
            plan = KVPlan.empty(b, capacity, ctx_len.device)
        else:
            with _on(stream):
                plan = KVPlan.empty(b, capacity, ctx_len.device)
    else:
        _ints(plan.row_start, "plan.row_start")
        _ints(plan.slots, "plan.slots", torch.int64)
        for name in ("positions", "request", "info"):
            _ints(getattr(plan, name), f"plan.{name}")
        _check(plan.row_start.shape[0] == b + 1 and plan.info.shape[0] == 4 and
               all(t.shape[0] >= capacity for t in plan[1:4]), "plan: buffers too small")
    row_start, slots, positions, request, info = plan
    _done("tern_kv_plan", B.lib().tern_kv_plan(
        ctx_len.data_ptr(), new_len.data_ptr(), b, page_size, table.data_ptr(), stride, width,
        free_pages.data_ptr(), free_pages.shape[0],
        None if free_head is None else free_head.data_ptr(), row_start.data_ptr(), capacity,
        slots.data_ptr(), positions.data_ptr(), request.data_ptr(), info.data_ptr(),
        B._stream(stream)))
    return plan


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """Rows of keys and values [T, heads, dim] into the cache's slots (-1: skipped)."""
    kt, kh = _heads(k, cache.heads, cache.dim, cache.dtype, "k")
    vt, vh = _heads(v, cache.heads, cache.dim, cache.dtype, "v")
    _ints(slots, "slots", torch.int64)
    t = k.shape[0]
    _check(v.shape[0] == t and slots.shape[0] >= t, "v, slots: expected as many rows as k")
    _done("tern_kv_write", B.lib().tern_kv_write(
        cache.address, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), t,
        B._stream(stream)))


def tree_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, ctx_len: torch.Tensor,
                   row_start: torch.Tensor, max_new: int, mask: torch.Tensor | None = None,
                   scale: float | None = None, out: torch.Tensor | None = None,
                   return_lse: bool = False, lse: torch.Tensor | None = None,
                   ws: B.Workspace | None = None, stream=None):
    """Attention of the new rows q [T, query heads, dim] over the paged cache:
    each row sees its request's ctx_len cached tokens and, of the request's
    new tokens (at most ``max_new`` <= 256 of them, already written), those
    whose bits are set in ``mask`` (int64 [T, words]; None: a chain, token i
    sees 0 .. i).  Returns out [T, query heads, dim], and with ``return_lse``
    also the logarithm of each row's sum of exponentials (fp32 [T, query heads]).
    A row that sees nothing is 0, its lse -infinity."""
    b = ctx_len.shape[0]
    t, hq, _ = q.shape
    heads, dim, dtype = cache.heads, cache.dim, cache.dtype
    qt, qh = _heads(q, hq, dim, dtype, "q")
    _check(hq > 0 and hq % heads == 0, "q: expected a multiple of the cache's heads")
    _ints(ctx_len, "ctx_len")
    _ints(row_start, "row_start")
    _check(row_start.shape[0] == b + 1, "row_start: expected one more entry than requests")
    stride, width = _table(table, b)
    words = 0
    if mask is not None:
        _ints(mask, "mask", torch.int64, 2)
        rows, words = mask.shape
        _check(rows >= t and words > 0, "mask: expected [rows, words]")
    if out is not None:
        _check(out.is_cuda and out.dtype is dtype and out.shape == (t, hq, dim) and
               out.is_contiguous(), "out: expected a contiguous [rows, query heads, dim]")
    if lse is not None:
        _check(lse.is_cuda and lse.dtype is torch.float32 and lse.shape == (t, hq) and
               lse.is_contiguous(), "lse: expected a contiguous fp32 [rows, query heads]")
    if stream is not None and (out is None or ws is None or (return_lse and lse is None)):
        with _on(stream):          # what is allocated here belongs to that stream
            return tree_attention(q, cache, table, ctx_len, row_start, max_new, mask, scale, out,
                                  return_lse, lse, ws)
    if out is None:
        out = torch.empty((t, hq, dim), dtype=dtype, device=cache.device)
    if return_lse and lse is None:
        lse = torch.empty((t, hq), dtype=torch.float32, device=cache.device)
    nb = _workspace_bytes(max_new, hq, heads, dim)
    if ws is None:
        ws = B.Workspace(cache.device)
    buf = ws.head(nb, B.TERN_TREE_ATTENTION_ZERO_BYTES, stream)
    _done("tern_tree_attention", B.lib().tern_tree_attention(
        q.data_ptr(), qt, qh, cache.address, table.data_ptr(), stride, width, ctx_len.data_ptr(),
        row_start.data_ptr(), None if mask is None else mask.data_ptr(), words, b, t, hq, max_new,
        dim ** -0.5 if scale is None else scale, out.data_ptr(),
        None if lse is None else lse.data_ptr(), buf.data_ptr(), buf.numel(), B._stream(stream)))
    return (out, lse) if return_lse else out


def kv_commit(caches: KVCache | Sequence[KVCache], table: torch.Tensor, ctx_len: torch.Tensor,
              path: torch.Tensor, path_len: torch.Tensor, ctx_out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Keep the accepted path of every request: the token path[b][j] of its
    new ones moves to place j behind its ctx_len[b] cached tokens, for
    j < path_len[b] and in every layer's cache.  Returns the new lengths.  A
    path has to increase; it is cut where it does not."""
    if isinstance(caches, KVCache):
        caches = (caches,)
    _check(len(caches) > 0, "caches: expected at least one")
    b = ctx_len.shape[0]
    _ints(ctx_len, "ctx_len")
    _ints(path_len, "path_len")
    _ints(path, "path", torch.int32, 2)
    _check(path.shape[0] == b and path_len.shape[0] == b, "path, path_len: expected a row each request")
    stride, width = _table(table, b)
    if ctx_out is None:
        if stream is None:
            ctx_out = torch.empty(b, dtype=torch.int32, device=ctx_len.device)
        else:
            with _on(stream):
                ctx_out = torch.empty(b, dtype=torch.int32, device=ctx_len.device)
    else:
        _ints(ctx_out, "ctx_out")
        _check(ctx_out.shape[0] == b, "ctx_out: expected as many requests as ctx_len")
    _done("tern_kv_commit", B.lib().tern_kv_commit(
        b"".join([c.desc_bytes for c in caches]), len(caches), table.data_ptr(), stride, width,
        ctx_len.data_ptr(), path.data_ptr(), path.shape[1], path_len.data_ptr(),
        ctx_out.data_ptr(), b, B._stream(stream)))
    return ctx_out


def ancestor_masks(parents: Sequence[int], device="cuda") -> torch.Tensor:
    """The mask of a drafted tree, int64 [tokens, words]: each token sees
    itself and its ancestors.  parents[i] < i is token i's parent (-1: it
    follows the cached tokens)."""
    words = max(1, -(-len(parents) // 64))
    rows = []
    for i, p in enumerate(parents):
        _check(-1 <= p < i, "parents: expected -1 or an earlier token")
        rows.append((1 << i) | (rows[p] if p >= 0 else 0))
    signed = [[((r >> (64 * w)) & (2 ** 64 - 1)) for w in range(words)] for r in rows]
    signed = [[x - 2 ** 64 if x >= 2 ** 63 else x for x in row] for row in signed]
    return torch.tensor(signed, dtype=torch.int64, device=device).reshape(len(parents), words)
