"""The sampler's weights one by one: rows whose drawn token depends on a weight's last bits."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import sampling
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("left_out", [0, 7])
@pytest.mark.parametrize("dtype,most,t,x", [
    (dtype, most, t, x) for dtype in (BF, HF, F32) for most, t in ((72.0, 6.0), (96.0, 8.0))
    for x in (136 * 2.0 ** -21, 2.0 ** -18)])
def test_weight_of_logits_far_smaller_than_the_largest(dtype, most, t, x, left_out):
    """One logit `most` and n of x, which 32 bits cannot subtract exactly: it is half a step, 2^-18, off.  (Some more
    that top-k leaves out.)  With r = exp((x - most) / t) the token is 1 + floor(f), f = (u (1 + n r) - 1) / r.  A
    relative error e of the weight moves f by (1 - u) e / r, so with 2^-28, or 2^-44 of the largest, 2^-44 / r, for e,
    those u are looked for whose f is further from a whole number than twice that, and nearer than the half step
    would move it."""
    n = 200000
    r = np.exp((x - most) / t)
    u = np.random.default_rng(int(most)).uniform(0.5, 0.95, 200000).astype(np.float32)
    f = (u.astype(np.float64) * (1 + n * r) - 1) / r
    away, each = np.abs(f - np.round(f)), (1 - u) / r
    take = (f > 0) & (away > 2 * each * (2.0 ** -28 + 2.0 ** -44 / r)) & (away < 0.6 * each * 2.0 ** -18 / t)
    u, f = u[take][:64], f[take][:64]
    assert len(u) == 64
    logits = torch.full((64, 1 + n + left_out), x, dtype=dtype, device="cuda")
    assert float(logits[0, 0]) == x
    logits[:, 0] = most
    top_k = torch.full((64,), 1 + n, dtype=torch.int32, device="cuda") if left_out else None
    token = sampling.sample(logits, torch.from_numpy(u).cuda(), temperature=torch.full((64,), t, device="cuda"),
                            top_k=top_k)
    assert np.array_equal(token.cpu().numpy(), np.floor(f).astype(np.int64) + 1)
