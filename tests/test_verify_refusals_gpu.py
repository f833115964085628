"""Steps of the verification stack that are refused or do not fit."""

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import verify as V
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

HIDDEN = 1024


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(pages=20):
    return V.random_stack(2, HIDDEN, 16, 4, 64, pages=pages, page_size=16, requests=2, width=24, seed=3)


def states(rows, seed=5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16)


REFUSED = [
    ("a prompt longer than a step takes", 320, 300, ints, torch.bfloat16, ValueError),
    ("hidden states of another type", 40, 20, ints, torch.float32, ValueError),
    ("a mask of another type", 40, 20, ints, torch.bfloat16, ValueError),
]


@pytest.mark.parametrize("what,rows,longest,lengths,dtype,error", REFUSED, ids=[r[0] for r in REFUSED])
def test_a_refused_step_leaves_the_stack_as_it_was(what, rows, longest, lengths, dtype, error):
    s, fresh = make(), make()
    for t in (s, fresh):
        t.step(states(30), ints([18, 12]), 18)
        t.commit(ints([list(range(18))] * 2), ints([18, 12]))
    before = (s.held.tolist(), s.free_head.tolist(), s.ctx_len.tolist())
    mask = torch.zeros(rows, 1, dtype=torch.int32, device="cuda") if "mask" in what else None
    with pytest.raises(error):
        s.step(states(rows).to(dtype), ints([rows - longest, longest]), longest, mask)
    assert (s.held.tolist(), s.free_head.tolist(), s.ctx_len.tolist()) == before
    # what follows is what follows without it, pages included
    for _ in range(2):
        x = states(40, seed=6)
        got, want = (t.step(x, ints([17, 23]), 23) for t in (s, fresh))
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        for t in (s, fresh):
            t.check()
            t.commit(ints([[0, 1, 2]] * 2), ints([3, 3]))
        assert s.held.tolist() == fresh.held.tolist() and s.free_head.tolist() == fresh.free_head.tolist()
    B.tern_check()


def test_a_step_that_does_not_fit_is_said():
    s = make(pages=3)
    s.step(states(30), ints([18, 12]), 18)
    s.check()
    s.commit(ints([list(range(18))] * 2), ints([18, 12]))
    s.step(states(40), ints([20, 20]), 20)              # no page is left
    with pytest.raises(RuntimeError, match="pages"):
        s.check()
    # a path is cut where its token has no page
    assert s.commit(ints([list(range(20))] * 2), ints([20, 20])).tolist() == [32, 16]
    with pytest.raises(RuntimeError, match="rows"):
        t = make()
        t.step(states(10), ints([20, 20]), 20)
        t.check()
