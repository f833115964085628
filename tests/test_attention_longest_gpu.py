"""The longest context that a block table can describe: positions up to the last of 31 bits."""

import math

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 16), (128, 128)])
def test_a_context_of_all_positions(dim, group):
    """Every page of the table but the last is the same one: keys of score 0 and values of 1.  The
    last one's eight keys score 21.5, about the logarithm of the others' number, with values of 3;
    the last two of them are the new tokens, a chain.

    Bounds: the counts are sums of whole numbers below 2^24 in every accumulator; the probabilities
    and the output are rounded to bf16 (2^-8 each), lse is a number below 32 in 32 bits, after a few
    roundings of 2^-24 and the exponential's 2^-21."""
    ensure_lib()
    page, width = 8, 2 ** 28 - 1
    cache = kv.KVCache.empty(2, page, 1, dim)
    cache.k.zero_()
    cache.k[1, :, :, 0] = 21.5
    cache.v[0], cache.v[1] = 1.0, 3.0
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.zeros(2, group, dim, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    out, lse = kv.tree_attention(q, cache, table, ints([width * page - 2]), ints([0, 2]), 2, scale=1.0,
                                 return_lse=True)
    B.tern_check()
    for i in range(2):
        plain, top = float((width - 1) * page), (7 + i) * math.exp(21.5)
        ref = (plain + 3 * top) / (plain + top)
        assert ((out[i].double() - ref).abs() <= 2.5 * 2.0 ** -8 * ref).all(), (out[i].unique(), ref)
        assert ((lse[i].double() - math.log(plain + top)).abs() <= 2.0 ** -17).all(), (lse[i].unique(), plain + top)
