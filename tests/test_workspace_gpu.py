"""Workspaces on a stream of their own and in graphs."""

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu

ZERO = B.TERN_TREE_ATTENTION_ZERO_BYTES


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("ask", [lambda ws, n, s: ws.head(n, ZERO, s), lambda ws, n, s: ws.get(n, s),
                                 lambda ws, n, s: ws.scratch(n, s)])
@pytest.mark.parametrize("handle", [False, True])
def test_a_buffer_that_was_outgrown_stays_with_its_stream(ask, handle):
    """The other stream may still use it, so the current stream must not be given its memory."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    torch.cuda.empty_cache()
    ws = B.Workspace()
    first = ask(ws, 3 << 20, stream).data_ptr()
    ask(ws, 64 << 20, stream)
    kept = [torch.empty(3 << 20, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert first not in [t.data_ptr() for t in kept]
    torch.cuda.synchronize()


def test_a_captured_call_leaves_the_workspace_to_be_zeroed():
    """A zero-fill that was captured has not run yet: a call before the graph's first replay needs its own."""
    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    gen = torch.Generator(device="cuda").manual_seed(2)
    cache = kv.KVCache.empty(64, 64, 2, 128)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    q = torch.randn(4, 4, 128, generator=gen, device="cuda").to(torch.bfloat16)
    table, ctx, start = ints([list(range(64))]), ints([4000]), ints([0, 4])
    want = kv.tree_attention(q, cache, table, ctx, start, 4)
    B.tern_check()
    ws, out = B.Workspace(), torch.empty_like(want)
    poison(ws.scratch(1 << 25))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.tree_attention(q, cache, table, ctx, start, 4, out=out, ws=ws)
    for run in (lambda: kv.tree_attention(q, cache, table, ctx, start, 4, out=out, ws=ws), graph.replay,
                lambda: kv.tree_attention(q, cache, table, ctx, start, 4, out=out, ws=ws), graph.replay):
        poison(out)
        run()
        B.tern_check()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_a_captured_zero_fill_is_not_taken_for_one_that_ran():
    ws = B.Workspace()
    poison(ws.scratch(1 << 20))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws.get(1 << 20)
    assert (ws.get(1 << 20) == 0).all() and ws.clean == 1 << 20
