"""Tokens from logits, and which drafts they accept: what ends a step of
decoding or of verifying drafts, between the model's last linear and
kv.kv_commit, over the C entry points.

Filters, random numbers, trees and results are device tensors, so a whole
step can be captured in a CUDA graph and replayed as they change.
"""

from __future__ import annotations

import contextlib

import torch

from . import binding as B
from . import kv

_TYPES = {torch.bfloat16: B.TERN_LOGITS_BF16, torch.float16: B.TERN_LOGITS_F16,
          torch.float32: B.TERN_LOGITS_F32}


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
           top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
           min_p: torch.Tensor | None = None, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """A token of each row of ``logits`` [rows, vocab] (bf16, fp16 or float32;
    rows may be apart), int32 [rows], from the random numbers ``u`` float32
    [rows] in [0, 1).

    Each row has its own filters, float32 [rows] (``top_k`` int32): a
    ``temperature`` of 0 takes the largest logit; then the ``top_k`` largest
    logits are kept (0: all), of those the tokens at least ``min_p`` times as
    likely as the first (0: all), and of those the fewest of the likeliest that
    hold ``top_p`` of the probability (1: all).  Of equal logits the lowest
    index comes first.  The token is the first, by index, at which the kept
    probabilities add to more than u.  -1: a row of -infinity only."""
    kv._check(logits.dtype in _TYPES, "logits: expected bf16, fp16 or float32")
    if out is None:
        with contextlib.nullcontext() if stream is None else B._on(stream):
            out = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
    st = (kv._calls or kv._native()).sample(logits, logits.dtype, _TYPES[logits.dtype], u, temperature,
                                            top_k, top_p, min_p, out, B._stream(stream))
    if st:
        kv._failed("tern_sample", st)
    return out


def accept(tokens: torch.Tensor, target: torch.Tensor, parents: torch.Tensor, row_start: torch.Tensor,
           max_new: int, path: torch.Tensor | None = None, path_len: torch.Tensor | None = None,
           next: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The drafts that the sampled tokens agree with, as kv.kv_commit takes
    them: ``path`` int32 [requests, max_new] (-1 behind its end), ``path_len``
    and ``next`` int32 [requests].

    A request's rows are row_start[b] .. (kv.kv_plan's): row 0 is its last
    known token, the others drafts with ``parents`` int32 [rows] among them
    (a row's is lower than itself).  ``tokens`` are the rows' own, ``target``
    those that were sampled behind each.  From row 0 the path goes on to the
    lowest row whose parent is the one before and whose token is that one's
    target; ``next`` is the target of its last row, a token that needs no
    further check.  A chain's parents are -1, 0, 1, ..."""
    if path is None or path_len is None or next is None:
        b = max(row_start.shape[0] - 1, 0)

        def ints(given, *shape):
            return torch.empty(shape, dtype=torch.int32, device=tokens.device) if given is None else given
        with contextlib.nullcontext() if stream is None else B._on(stream):
            path, path_len, next = ints(path, b, max_new), ints(path_len, b), ints(next, b)
    kv._check(path.ndim == 2 and path.shape[1] == max_new, "path: expected [requests, max_new]")
    st = (kv._calls or kv._native()).accept(tokens, target, parents, row_start, path, path_len, next,
                                            B._stream(stream))
    if st:
        kv._failed("tern_tree_accept", st)
    return path, path_len, next
