"""Steps whose pages run out: what a request is said to hold is what it got, and a later step
with pages again fills what was missing."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import kv
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def held_after(ctx, new, page, width, held, left):
    """Pages in each table row after a step with ``left`` free pages."""
    out = []
    for c, n, h in zip(ctx, new, held):
        got = min(max(min(-(-(c + n) // page), width) - h, 0), left)
        out.append(h + got)
        left -= got
    return out


def test_pages_that_ran_out_are_taken_by_the_next_step():
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    held, out, after = ints([0, 0, 0]), poison(ints([0] * 3)), poison(ints([0] * 3))
    new = ints([20, 40, 17])                       # 2, 3 and 2 pages of 16, of which there are four
    first = kv.kv_plan(ints([0, 0, 0]), new, table, ints([7, 8, 9, 10]), 16, 77, held=held, held_out=out)
    assert first.info.tolist() == [77, 4, 4, 1]
    assert table.tolist() == [[7, 8, -1, -1], [9, 10, -1, -1], [-1, -1, -1, -1]]
    assert out.tolist() == [2, 2, 0]
    # the same tokens again, with pages
    second = kv.kv_plan(ints([0, 0, 0]), new, table, ints([3, 4, 5]), 16, 77, held=out, held_out=after)
    assert table.tolist() == [[7, 8, -1, -1], [9, 10, 3, -1], [4, 5, -1, -1]]
    assert after.tolist() == [2, 3, 2] and second.info.tolist() == [77, 3, 3, 0]
    assert min(second.slots.tolist()) >= 0 and len(set(second.slots.tolist())) == 77


@pytest.mark.parametrize("requests", [5, 513, 1500])
def test_what_is_held_after_steps_that_run_out(requests):
    rng = np.random.default_rng(requests)
    page, width, steps = 8, 6, 4
    ctx = rng.integers(0, 20, requests)
    held = -(-ctx // page)
    table = np.full((requests, width), -1)
    for b, h in enumerate(held):
        table[b, :h] = 100000 + 10 * b + np.arange(h)
    table, at = ints(table.tolist()), ints(held.tolist())
    next_page = 0
    for step in range(steps):
        new = rng.integers(0, 24, requests)
        free = int(rng.integers(0, requests))
        pages = list(range(next_page, next_page + free))
        next_page += free
        out = poison(torch.empty(requests, dtype=torch.int32, device="cuda"))
        got = kv.kv_plan(ints(ctx.tolist()), ints(new.tolist()), table, ints(pages), page, int(new.sum()),
                         held=at, held_out=out)
        want = held_after(ctx, new, page, width, held, free)
        assert out.tolist() == want
        rows = table.tolist()
        assert all(rows[b][j] >= 0 for b in range(requests) for j in range(want[b]))
        # a row has a slot where its page is held, and nowhere else
        slots, row = got.slots.tolist(), 0
        for b in range(requests):
            for i in range(new[b]):
                p = int(ctx[b]) + i
                known = p // page < want[b]
                assert slots[row] == (rows[b][p // page] * page + p % page if known else -1)
                row += 1
        held, at = np.asarray(want), out
