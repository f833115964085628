"""Requests with more new tokens than the call was told of, at sizes where a row's number is large."""

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu


def test_more_tokens_than_said_with_many_query_heads_on_a_key_head():
    """1040 tokens of 2048 query heads on each of two key heads: 2^21 rows on a key head and
    more, each of which has to be written in its own place and nothing behind the last."""
    ensure_lib()
    tokens, heads, group, dim, page = 1040, 2, 2048, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache = kv.KVCache.empty(1, page, heads, dim)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    q = torch.randn(tokens, heads * group, dim, generator=gen, device="cuda", dtype=torch.bfloat16)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    whole = poison(torch.empty(tokens + 16, heads * group, dim, dtype=torch.bfloat16, device="cuda"))
    # a table of one page: eight keys, of which token i sees 0 .. i
    kv.tree_attention(q, cache, ints([[0]]), ints([0]), ints([0, tokens]), 1, out=whole[:tokens])
    B.tern_check()
    assert (whole[tokens:].view(torch.int16) == -1).all()
    i, j = torch.arange(tokens, device="cuda")[:, None], torch.arange(page, device="cuda")
    for h in range(heads):
        s = q[:, h * group:(h + 1) * group].double() @ cache.k[0, :, h].double().T * dim ** -0.5
        p = s.masked_fill((j > i)[:, None, :], float("-inf")).softmax(-1)
        v = cache.v[0, :, h].double()
        ref, weight = p @ v, p @ v.abs()
        got = whole[:tokens, h * group:(h + 1) * group].double()
        # the probabilities' and the output's rounding (2^-8 each), with half as much again for 32-bit sums
        assert ((got - ref).abs() <= 1.5 * 2.0 ** -8 * (weight + ref.abs())).all()
