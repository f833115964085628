"""The paged key/value cache and the verification of drafted-token trees.

What a decode step that verifies drafted tokens needs between its qkv and its
output linear, over the C entry points of the same names:

* ``kv_plan``: block tables and slot maps on the GPU from the requests' lengths;
* ``kv_write``: the new tokens' keys and values into the cache;
* ``tree_attention``: every row over its request's cached tokens and, of the
  request's new tokens, those that its mask names;
* ``kv_commit``: the accepted path of each tree made contiguous, all layers.

The cache holds 16-bit values (``KVCache``) or 8-bit codes with a unit for
each row (``KVCache8``, ``kv_read``); the same calls take both.  ``rotate_write`` writes rows as
``kv_write`` does, with the norms of queries and keys and their rotary
positions in the same pass.

Lengths, tables, masks and paths are device tensors that only the kernels
read, so a step can be captured in a CUDA graph and replayed as they change.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import importlib.util
import math
import os
from fractions import Fraction
from typing import NamedTuple, Sequence

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.TERN_KV_BF16, torch.float16: B.TERN_KV_F16}
_CODES = {torch.int8: B.TERN_KV_I8, torch.float8_e4m3fn: B.TERN_KV_E4M3}


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

        def at(*names):
            return [ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names]
        module.bind(*at(*names), torch.int32, torch.int64, torch.float32,
                    torch._C._cuda_getDevice if _several_devices() else None)
        module.bind8(*at("tern_kv_rotate_write", "tern_kv8_read", "tern_kv8_commit", "tern_tree_attention8"))
        module.bind_tokens(*at("tern_sample", "tern_tree_accept"))
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
def _workspace_bytes(max_new: int, hq: int, heads: int, dim: int, index: int, eight: bool) -> int:
    if eight:
        return B.tern_tree_attention8_workspace_bytes(max_new, hq, heads, dim)
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


class KVCache8:
    """Keys and values of one layer in 8 bits: ``k`` and ``v`` [pages,
    page_size, heads, dim] of int8 or float8_e4m3fn as for KVCache, and a
    unit for each token and head, ``k_scale`` and ``v_scale`` float32 [pages,
    heads, page_size] with the same strides (dense along the last axis).  A
    value is its code times its row's unit; written, a row's unit is its
    largest magnitude divided by 127 or 448.

    int8 keeps all of a row's values to 1/254 of the largest, e4m3 each to
    1/16 of itself: the first is more exact by a factor of about four unless a
    few channels are much larger than the others."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _check(k.is_cuda and k.ndim == 4 and k.dtype in _CODES,
               "k: expected a 4-D CUDA tensor of int8 or float8_e4m3fn")
        _check(v.is_cuda and v.device == k.device and v.dtype == k.dtype and v.shape == k.shape and
               v.stride() == k.stride(), "v: expected the device, type, shape and strides of k")
        _check(k.stride(3) == 1, "k, v: expected to be dense along the last axis")
        self.pages, self.page_size, self.heads, self.dim = k.shape
        for t in (k_scale, v_scale):
            _check(t.is_cuda and t.device == k.device and t.dtype == torch.float32 and
                   t.shape == (self.pages, self.heads, self.page_size) and
                   t.stride() == k_scale.stride() and t.stride(2) == 1,
                   "k_scale, v_scale: expected float32 [pages, heads, page_size] on k's device, "
                   "dense along the last axis")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        # an axis of length one may have any stride: give it one that passes
        ps, ts, hs = (k.stride(i) if k.shape[i] > 1 else self.page_size * self.heads * self.dim
                      for i in range(3))
        sp, sh = (k_scale.stride(i) if k_scale.shape[i] > 1 else self.page_size * self.heads
                  for i in range(2))
        self.desc = B.KVCache8Desc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   self.pages, self.page_size, self.heads, self.dim, ps, ts, hs, sp, sh,
                                   _CODES[k.dtype])
        self.desc_bytes = bytes(self.desc)
        self.address = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int, dtype=torch.int8, device="cuda",
              heads_first: bool = False) -> "KVCache8":
        """A cache of uninitialised pages, rows of heads or (``heads_first``) heads of rows."""
        if heads_first:
            k, v = (torch.empty((pages, heads, page_size, dim), dtype=dtype, device=device)
                    .transpose(1, 2) for _ in range(2))
        else:
            k, v = (torch.empty((pages, page_size, heads, dim), dtype=dtype, device=device)
                    for _ in range(2))
        units = (torch.empty((pages, heads, page_size), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, *units)


# 1 / (2 pi), to 2^-120
_TURNS = Fraction(10 ** 40, 62831853071795864769252867665590057683943)


class Rotary:
    """Rotary positions: pair j of a head's first 2 * len(freq) elements (a
    multiple of 16; the others stay) is turned by position * freq[j] radians.
    ``axis`` [pairs] says which of several positions of a token turns each
    pair, e.g. time, height and width of an image's tokens.  Pairs are (j, j +
    pairs), or with ``neighbours`` (2 j, 2 j + 1).  ``freq``, numbers or a tensor
    of them, is read once; a scaling of long contexts that changes angles goes
    into it.  One that also multiplies cosines and sines by a factor is said
    elsewhere: its square in the attention's ``scale`` where all of a head is
    rotated, or the factor in the rotated elements of ``q_norm`` and ``k_norm``."""

    def __init__(self, freq, axis=None, neighbours: bool = False, device="cuda"):
        if isinstance(freq, torch.Tensor):
            device = freq.device if freq.is_cuda else device
            freq = freq.tolist()
        if isinstance(axis, torch.Tensor):
            axis = axis.tolist()
        _check(len(freq) > 0 and len(freq) % 8 == 0 and all(math.isfinite(f) for f in freq),
               "freq: expected a multiple of 8 finite numbers")
        _check(axis is None or (len(axis) == len(freq) and min(axis) >= 0),
               "axis: expected a number each of freq")
        # turns a position as a 64-bit fraction: of an angle only what is past whole turns counts
        turn = [int(Fraction(f) * _TURNS * 2 ** 64) % 2 ** 64 for f in freq]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turn], dtype=torch.int64,
                                  device=device)
        self.axes = 1 if axis is None else max(axis) + 1
        self.axis = None if axis is None else torch.tensor(axis, dtype=torch.int32, device=device)
        self.rot, self.neighbours = 2 * len(freq), bool(neighbours)

    @classmethod
    def geometric(cls, rot: int, base: float = 1e6, **kw) -> "Rotary":
        """The usual frequencies of ``rot`` elements, base^(-2 j / rot)."""
        return cls([base ** (-2 * j / rot) for j in range(rot // 2)], **kw)


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


def kv_write(cache: KVCache | KVCache8, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """Rows of keys and values [T, heads, dim] into the cache's slots (-1: skipped);
    bf16 or fp16 rows are quantised on their way into an 8-bit cache."""
    if isinstance(cache, KVCache8):
        rotate_write(cache, None, k, v, slots, stream=stream)
        return
    st = (_calls or _native()).write(cache.address, cache.dtype, cache.heads, cache.dim,
                                     cache.index, k, v, slots, B._stream(stream))
    if st:
        _failed("tern_kv_write", st)


def rotate_write(cache: KVCache | KVCache8, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                 slots: torch.Tensor, rotary: Rotary | None = None, positions: torch.Tensor | None = None,
                 q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, eps: float = 1e-6,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """kv_write with what comes before it, in one pass: queries [T, query
    heads, dim] and keys divided by their root mean square of each head and
    multiplied by ``q_norm`` and ``k_norm`` [dim] (of the rows' type or both
    float32; None: no norm), then turned by ``rotary`` at ``positions``, int32
    [T], or [axes, T] where it has several axes.  Returns the queries (``out``,
    which may be q itself where that is contiguous).  All of it is in 32 bits
    and rounded once."""
    dtype, eight = k.dtype, isinstance(cache, KVCache8)
    _check(dtype in _TYPES, "k: expected bf16 or fp16")
    _check(eight or dtype == cache.dtype, "k: expected the cache's type")
    if q is not None and out is None:
        with contextlib.nullcontext() if stream is None else B._on(stream):
            out = torch.empty(q.shape, dtype=dtype, device=cache.device)
    several, turns, axis, neighbours = False, None, None, False
    if rotary is not None:
        _check(positions is not None, "positions: expected with rotary")
        several = positions.ndim == 2
        turns, axis, neighbours = rotary.turns, rotary.axis, rotary.neighbours
        _check(rotary.axes == 1 or (several and positions.shape[0] >= rotary.axes),
               "positions: expected [axes, rows], as rotary has several axes")
        _check(rotary.rot <= cache.dim, "rotary: expected no more elements than a head has")
    norm = q_norm if q_norm is not None else k_norm
    norm = dtype if norm is None else norm.dtype
    _check(norm in (dtype, torch.float32), "q_norm, k_norm: expected the rows' type or float32")
    st = (_calls or _native()).rotate(
        0 if eight else cache.address, cache.address if eight else 0, dtype, _TYPES[dtype], cache.heads,
        cache.dim, cache.index, q, k, v, slots, positions, several, turns, axis, neighbours, q_norm,
        k_norm, norm, eps, out, B._stream(stream))
    if st:
        _failed("tern_kv_rotate_write", st)
    return out


def kv_read(cache: KVCache8, slots: torch.Tensor, dtype=torch.bfloat16, k: torch.Tensor | None = None,
            v: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The rows in ``slots`` of an 8-bit cache as 16-bit values: keys and
    values [T, heads, dim] (zeros for a slot outside the cache)."""
    _check(isinstance(cache, KVCache8), "cache: expected an 8-bit one")
    given = k if k is not None else v
    if given is not None:
        dtype = given.dtype
    _check(dtype in _TYPES, "dtype: expected bf16 or fp16")
    if k is None or v is None:
        shape = (slots.shape[0] if given is None else given.shape[0], cache.heads, cache.dim)
        with contextlib.nullcontext() if stream is None else B._on(stream):
            k = torch.empty(shape, dtype=dtype, device=cache.device) if k is None else k
            v = torch.empty(shape, dtype=dtype, device=cache.device) if v is None else v
    st = (_calls or _native()).read(cache.address, cache.heads, cache.dim, cache.index, slots, dtype,
                                    _TYPES[dtype], k, v, B._stream(stream))
    if st:
        _failed("tern_kv8_read", st)
    return k, v


def tree_attention(q: torch.Tensor, cache: KVCache | KVCache8, table: torch.Tensor, ctx_len: torch.Tensor,
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
    else up to the output's own rounding is in 32 bits.

    Over an 8-bit cache q is bf16 or fp16, and out of its type; codes enter the
    products as they are, and probabilities times the values' units are rounded
    to fp16."""
    t, hq, _ = q.shape
    heads, dim, eight = cache.heads, cache.dim, isinstance(cache, KVCache8)
    dtype = q.dtype if eight else cache.dtype
    _check(dtype in _TYPES, "q: expected bf16 or fp16")
    if stream is not None and (out is None or ws is None or (return_lse and lse is None)):
        with B._on(stream):          # what is allocated here belongs to that stream
            return tree_attention(q, cache, table, ctx_len, row_start, max_new, mask, scale, out,
                                  return_lse, lse, ws)
    if out is None:
        out = torch.empty((t, hq, dim), dtype=dtype, device=cache.device)
    if return_lse and lse is None:
        lse = torch.empty((t, hq), dtype=torch.float32, device=cache.device)
    need, at, size = _workspace_bytes(max_new, hq, heads, dim, cache.index, eight), 0, 0
    if need:      # none: there are no new tokens, or the call below refuses what it gets
        buf = (B.Workspace(cache.device) if ws is None else ws).head(
            need, B.TERN_TREE_ATTENTION_ZERO_BYTES, stream)
        _check(buf.get_device() == cache.index, "ws: expected a workspace on the cache's device")
        at, size = buf.data_ptr(), buf.numel()
    calls = _calls or _native()
    args = (cache.address, dtype, heads, dim, cache.index, q, table, ctx_len, row_start, max_new, mask,
            dim ** -0.5 if scale is None else scale, out, lse, at, size, B._stream(stream))
    st = calls.attention8(*args, _TYPES[dtype]) if eight else calls.attention(*args)
    if st:
        _failed("tern_tree_attention8" if eight else "tern_tree_attention", st)
    return (out, lse) if return_lse else out


def kv_commit(caches: KVCache | KVCache8 | Sequence[KVCache | KVCache8], table: torch.Tensor, ctx_len: torch.Tensor,
              path: torch.Tensor, path_len: torch.Tensor, ctx_out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Keep the accepted path of every request: the token path[b][j] of its
    new ones moves to place j behind its ctx_len[b] cached tokens, for
    j < path_len[b] and in every layer's cache.  Returns the new lengths.  A
    path has to increase; it is cut where it does not."""
    if isinstance(caches, (KVCache, KVCache8)):
        caches = (caches,)
    _check(len(caches) > 0 and (not _several_devices() or len({c.index for c in caches}) == 1),
           "caches: expected one or more, on the same device")
    eight = isinstance(caches[0], KVCache8)
    _check(all(isinstance(c, KVCache8) == eight for c in caches), "caches: expected all of 16 bits or all of 8")
    if ctx_out is None:
        if stream is None:
            ctx_out = torch.empty(ctx_len.shape[0], dtype=torch.int32, device=ctx_len.device)
        else:
            with B._on(stream):
                ctx_out = torch.empty(ctx_len.shape[0], dtype=torch.int32, device=ctx_len.device)
    calls = _calls or _native()
    st = (calls.commit8 if eight else calls.commit)(
        b"".join([c.desc_bytes for c in caches]), len(caches), caches[0].index, table, ctx_len, path,
        path_len, ctx_out, B._stream(stream))
    if st:
        _failed("tern_kv8_commit" if eight else "tern_kv_commit", st)
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
