"""The cache's calls on a stream given by its handle, the default stream's 0 among them."""

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("form", ["default handle", "default", "side handle", "side"])
def test_calls_come_behind_what_their_stream_has_to_do(form):
    stream = torch.cuda.Stream() if form.startswith("side") else torch.cuda.default_stream()
    gen = torch.Generator(device="cuda").manual_seed(4)
    cache = kv.KVCache.empty(8, 16, 2, 64)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    q = torch.randn(3, 4, 64, generator=gen, device="cuda").to(torch.bfloat16)
    table, start, free = ints([[0, 1, 2, 3]]), ints([0, 3]), ints([4, 5])
    path, path_len = ints([[0, 2]]), ints([2])
    want = kv.tree_attention(q, cache, table, ints([40]), start, 3, return_lse=True)
    want_plan = kv.kv_plan(ints([40]), ints([3]), table.clone(), free, 16, 3)
    ctx, late = ints([7]), ints([40])
    early, warm = torch.zeros_like(q), torch.cuda.Stream()
    kv.tree_attention(q, cache, table, ctx, start, 3, stream=warm)       # what a first call sets up
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)          # some 50 ms
        ctx.copy_(late)
        early.copy_(q)
    handle = stream.cuda_stream if form.endswith("handle") else stream
    assert form != "default handle" or handle == 0
    got = kv.tree_attention(early, cache, table, ctx, start, 3, return_lse=True, stream=handle)
    plan = kv.kv_plan(ctx, ints([3]), table.clone(), free, 16, 3, stream=handle)
    length = kv.kv_commit(cache, table, ctx, path, path_len, stream=handle)
    torch.cuda.synchronize()
    B.tern_check()
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    assert plan.slots.tolist() == want_plan.slots.tolist() and length.tolist() == [42]
