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
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Sequence

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.TERN_KV_BF16, torch.float16: B.TERN_KV_F16}


def _check(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


_calls = None


def _native():
    """The calls' checks and marshalling (csrc/kvcall.c, built with the library):
    in Python they cost more host time at decode sizes than the launch."""
    global _calls
    if _calls is None:
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_kvcall.so")
        if not os.path.exists(path):
            raise RuntimeError(f"_kvcall.so not built ({path}); run "
                               "ternary_weight_linear_block_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_kvcall", path)
        spec = importlib.util.spec_from_file_location("_kvcall", path, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        lib = B.lib()
        names = ("tern_kv_plan", "tern_kv_write", "tern_tree_attention", "tern_kv_commit")
        module.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names),
                    torch.int32, torch.int64, torch.float32,
                    torch._C._cuda_getDevice if _several_devices() else None)
        _calls = module
    return _calls


@functools.cache
def _several_devices() -> bool:
    """Whether a CUDA tensor can be on another device than the current one; where it
    cannot, asking costs a small call up to a microsecond for nothing."""
    return torch.cuda.device_count() > 1


def _failed(name: str, status: int):
    raise B.TernError(name, status)


@functools.lru_cache(maxsize=None)
def _workspace_bytes(max_new: int, hq: int, heads: int, dim: int, index: int) -> int:
    return B.tern_tree_attention_workspace_bytes(max_new, hq, heads, dim)


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
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
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
    positions: torch.Tensor   # int32 [capacity]: each row's place in its request's cache (see kv_plan)
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
            held: torch.Tensor | None = None, held_out: torch.Tensor | None = None,
            stream=None) -> KVPlan:
    """Block tables and slot maps of one step: request b gets new_len[b] rows
    behind its ctx_len[b] cached tokens; the pages that they need beyond
    those it has are taken from ``free_pages`` (from index free_head[0] on)
    and written into ``table`` in place.  ``capacity`` rows are planned;
    ``plan`` gives the outputs' buffers (slots, positions and request 16-byte
    aligned).  info[2] is the next step's free_head
    (steps that reuse buffers take turns with two), info[3] says what did not fit.

    ``positions`` are places in the cache, ctx_len + the row's index: of a
    prompt's or a chain's tokens also their positions, e.g. for a rotary
    embedding.  A tree's token has position ctx_len + tree_depths, which is
    the place that kv_commit moves it to.

    A request has the pages of its cached tokens, or ``held`` int32
    [requests] of them: the pages of drafts that were not kept stay in its
    table row, and ``held_out`` (another tensor) says how many it has now."""
    if plan is None:
        if stream is None:
            plan = KVPlan.empty(ctx_len.shape[0], capacity, ctx_len.device)
        else:
            with B._on(stream):
                plan = KVPlan.empty(ctx_len.shape[0], capacity, ctx_len.device)
    st = (_calls or _native()).plan(ctx_len, new_len, table, free_pages, free_head, page_size,
                                    capacity, *plan, held, held_out, B._stream(stream))
    if st:
        _failed("tern_kv_plan", st)
    return plan


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """Rows of keys and values [T, heads, dim] into the cache's slots (-1: skipped)."""
    st = (_calls or _native()).write(cache.address, cache.dtype, cache.heads, cache.dim,
                                     cache.index, k, v, slots, B._stream(stream))
    if st:
        _failed("tern_kv_write", st)


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
    A row that sees nothing is 0, its lse -infinity.  The probabilities are
    rounded to the cache's type for their product with the values; everything
    else up to the output's own rounding is in 32 bits."""
    t, hq, _ = q.shape
    heads, dim, dtype = cache.heads, cache.dim, cache.dtype
    if stream is not None and (out is None or ws is None or (return_lse and lse is None)):
        with B._on(stream):          # what is allocated here belongs to that stream
            return tree_attention(q, cache, table, ctx_len, row_start, max_new, mask, scale, out,
                                  return_lse, lse, ws)
    if out is None:
        out = torch.empty((t, hq, dim), dtype=dtype, device=cache.device)
    if return_lse and lse is None:
        lse = torch.empty((t, hq), dtype=torch.float32, device=cache.device)
    need, at, size = _workspace_bytes(max_new, hq, heads, dim, cache.index), 0, 0
    if need:      # none: there are no new tokens, or the call below refuses what it gets
        buf = (B.Workspace(cache.device) if ws is None else ws).head(
            need, B.TERN_TREE_ATTENTION_ZERO_BYTES, stream)
        _check(buf.get_device() == cache.index, "ws: expected a workspace on the cache's device")
        at, size = buf.data_ptr(), buf.numel()
    st = (_calls or _native()).attention(
        cache.address, dtype, heads, dim, cache.index, q, table, ctx_len, row_start, max_new, mask,
        dim ** -0.5 if scale is None else scale, out, lse, at, size, B._stream(stream))
    if st:
        _failed("tern_tree_attention", st)
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
    _check(len(caches) > 0 and (not _several_devices() or len({c.index for c in caches}) == 1),
           "caches: expected one or more, on the same device")
    if ctx_out is None:
        if stream is None:
            ctx_out = torch.empty(ctx_len.shape[0], dtype=torch.int32, device=ctx_len.device)
        else:
            with B._on(stream):
                ctx_out = torch.empty(ctx_len.shape[0], dtype=torch.int32, device=ctx_len.device)
    st = (_calls or _native()).commit(b"".join([c.desc_bytes for c in caches]), len(caches),
                                      caches[0].index, table, ctx_len, path, path_len, ctx_out,
                                      B._stream(stream))
    if st:
        _failed("tern_kv_commit", st)
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


def tree_depths(parents: Sequence[int], device="cuda") -> torch.Tensor:
    """How many ancestors each token of a drafted tree has, int32 [tokens]:
    its position is this much behind the cached tokens.  ``parents`` as for
    ancestor_masks."""
    depths = []
    for i, p in enumerate(parents):
        _check(-1 <= p < i, "parents: expected -1 or an earlier token")
        depths.append(depths[p] + 1 if p >= 0 else 0)
    return torch.tensor(depths, dtype=torch.int32, device=device)
