"""Attention whose result lies in many keys of small probability beside a few that dominate."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("below", [15.3, 20.6, 24.6, 26.2])
@pytest.mark.parametrize("requests,ctx", [(1, 60), (1, 2000), (320, 2000)])
@pytest.mark.parametrize("dim,group,new", [(64, 1, 1), (128, 4, 4), (256, 1, 3), (64, 4, 8), (128, 4, 8),
                                           (256, 4, 8), (128, 8, 20)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_keys_far_below_a_few(dtype, dim, group, new, requests, ctx, below):
    """The first 64 keys hold one of score 0 in every 16; all others score -``below`` in base 2,
    and alone have values.  The exact result: n v p / (d + n p) with p = 2^-below, n such keys and
    d dominant ones.  Both 16-bit types have to keep the probabilities' relative precision: fp16
    has no numbers below 2^-24 and few bits below 2^-14.

    Bounds: kv_reference.attention_bounds, whose weight is the result itself here, and for fp16's
    rounding of the probabilities at most 2^-32 a key of the largest (half the distance of its
    smallest numbers, 2^-25, where the largest is held as 2^7 or more)."""
    page, heads = 64, 1
    width = -(-(ctx + new) // page)
    cache = kv.KVCache.empty(width, page, heads, dim, dtype)
    cache.k.zero_()
    # scores: q = (1, 0, ..), k = (0 or -below, 0, ..) in the type, scale ln 2
    low = torch.tensor(-below).to(dtype).item()
    value = 1.5 * 2.0 ** 12                       # keeps the result in the type's normal range
    cache.k[:, :, :, 0] = low
    cache.v.fill_(value)
    top = [0, 16, 32, 48]
    for t in top:
        cache.k[0, t, :, 0] = 0
        cache.v[0, t] = 0
    q = torch.zeros((requests * new, heads * group, dim), dtype=dtype, device="cuda")
    q[:, :, 0] = 1
    table = ints([list(range(width))] * requests)         # the same pages for every request
    start = ints([new * b for b in range(requests + 1)])
    out, lse = kv.tree_attention(q, cache, table, ints([ctx] * requests), start, new, scale=float(np.log(2)),
                                 return_lse=True)
    B.tern_check()
    out, lse = (t.double().cpu().numpy().reshape(requests, new, -1) for t in (out, lse))
    for i in range(new):
        n, p = ctx + i + 1 - len(top), 2.0 ** low
        ref, ref_lse = n * value * p / (len(top) + n * p), np.log(len(top) + n * p)
        assert ref > 2.0 ** -14
        qn, kn = np.eye(1, dim), np.eye(1, dim) * low
        of_out, of_lse = R.attention_bounds(qn, kn, dim, ctx + new, float(np.log(2)), dtype, ref, ref, ref_lse)
        if dtype == torch.float16:
            of_out += n * value * 2.0 ** -32
        assert np.abs(out[:, i] - ref).max() <= of_out, (i, out[:, i].min(), out[:, i].max(), ref)
        assert np.abs(lse[:, i] - ref_lse).max() <= of_lse
