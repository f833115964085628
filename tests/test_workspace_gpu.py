"""Workspaces on a stream of their own."""

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from tests.gpu_helpers import ensure_lib

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
