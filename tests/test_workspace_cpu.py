"""What the workspace and the tree attention's call ask of the device, with the device's part
recorded in place of run (no GPU needed)."""

from types import SimpleNamespace

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import build as BUILD
from ternary_weight_linear_block_gb300 import kv

ZERO = B.TERN_TREE_ATTENTION_ZERO_BYTES


@pytest.fixture
def zeroed(monkeypatch):
    """The zero-fills that were asked for, as (bytes of the buffer, bytes to zero)."""
    calls = []
    monkeypatch.setattr(B, "tern_workspace_init",
                        lambda buf, nbytes, stream=None: calls.append((buf.numel(), nbytes)))
    return calls


@pytest.mark.parametrize("nbytes", [0, 1, 256, ZERO - 1, ZERO, ZERO + 1, 1 << 20])
def test_head_zeroes_within_its_buffer(zeroed, nbytes):
    for ws in (B.Workspace("cpu"), B.Workspace("cpu")):
        buf = ws.head(nbytes, ZERO)
        assert buf.numel() >= max(nbytes, ZERO)
        assert ws.head(nbytes, ZERO) is buf
    assert len(zeroed) == 2 and all(want <= have for have, want in zeroed), zeroed


def test_head_of_a_buffer_made_for_something_smaller(zeroed):
    ws = B.Workspace("cpu")
    ws.scratch(300)
    ws.head(0, ZERO)
    ws.scratch(10)
    ws.head(0, ZERO)
    assert len(zeroed) == 2 and all(want <= have for have, want in zeroed), zeroed


@pytest.mark.parametrize("max_new,hq,heads,dim", [
    (0, 4, 2, 64), (257, 4, 2, 64), (-1, 4, 2, 64), (300, 20, 20, 128), (4, 5, 2, 64), (4, 1, 2, 64),
    (4, 4, 2, 96)])
def test_attention_calls_without_work_or_refused_use_no_workspace(zeroed, monkeypatch, max_new, hq,
                                                                  heads, dim):
    """Such a call reaches the checks (here: recorded) without a workspace and with nothing zeroed."""
    BUILD.ensure_built()
    seen = []
    monkeypatch.setattr(kv, "_native", lambda: SimpleNamespace(attention=lambda *a: seen.append(a) or 2))
    monkeypatch.setattr(kv, "_calls", None)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    cache = SimpleNamespace(heads=heads, dim=dim, dtype=torch.bfloat16, device=torch.device("cpu"), index=0,
                            address=0)
    q, ints = torch.zeros(3, hq, dim, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    out = torch.empty_like(q)
    for ws in (None, B.Workspace("cpu")):
        with pytest.raises(B.TernError):
            kv.tree_attention(q, cache, ints.reshape(1, 2), ints[:1], ints, max_new, out=out, ws=ws)
    assert zeroed == [] and len(seen) == 2
