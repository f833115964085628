"""Positions of drafted tokens: a token of a tree stands behind its ancestors, wherever its row is."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from ternary_weight_linear_block_gb300 import verify as V
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 1024, 16, 4, 64, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def turn(x, positions):
    """A rotary embedding: pairs (i, i + DIM / 2) turned by position / 100^(2 i / DIM)."""
    rate = 100.0 ** (-torch.arange(DIM // 2, device=x.device) * 2.0 / DIM)
    angle = positions.float()[:, None, None] * rate
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(x.dtype)


class Turner:
    def __init__(self):
        self.positions = []

    def __call__(self, q, k, positions):
        self.positions.append(positions.tolist())
        return turn(q, positions), turn(k, positions)


def test_kept_drafts_stand_in_the_place_they_were_turned_for():
    s = V.random_stack(1, HIDDEN, HEADS, KV_HEADS, DIM, pages=40, page_size=PAGE, requests=2, width=12, seed=3)
    block, rotate = s.blocks[0], Turner()
    gen = torch.Generator(device="cuda").manual_seed(5)

    def states(rows):
        return torch.randn(rows, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16)

    def keys(x):
        qkv = B.forward(block.qkv, x)
        q, k = qkv[:, :HEADS * DIM], qkv[:, HEADS * DIM:(HEADS + KV_HEADS) * DIM]
        return q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM))

    def cached(b, place):
        return block.cache.k[int(s.table[b, place // PAGE]), place % PAGE]

    prompt, x = [21, 9], states(30)
    s.step(x, ints(prompt), 21, rotate=rotate)                    # a chain: a token's place is its position
    assert rotate.positions == [list(range(21)) + list(range(9))]
    s.commit(ints([list(range(21))] * 2), ints(prompt))
    turned = turn(keys(x)[1], ints(rotate.positions[0]))
    assert torch.equal(cached(0, 20), turned[20]) and torch.equal(cached(1, 8), turned[29])

    trees, paths = [[-1, 0, 0, 1, 2, 2], [-1, -1, 1, 1, 3]], [[0, 2, 5], [1, 3]]
    depths = [[0, 1, 1, 2, 2, 2], [0, 0, 1, 1, 2]]
    assert [kv.tree_depths(t, device="cpu").tolist() for t in trees] == depths
    depth = torch.cat([kv.tree_depths(t) for t in trees])
    mask = torch.cat([kv.ancestor_masks(t) for t in trees])
    x, ctx = states(11), list(prompt)
    y = s.step(x, ints([6, 5]), 6, mask, depth=depth, rotate=rotate)
    assert rotate.positions[1] == [21 + d for d in depths[0]] + [9 + d for d in depths[1]]
    # the step with keys and queries turned by hand
    where = ints(rotate.positions[1])
    q, k = (turn(t, where) for t in keys(x))
    assert torch.equal(block.cache.k[s.plan.slots // PAGE, s.plan.slots % PAGE], k)
    a = kv.tree_attention(q, block.cache, s.table, s.ctx_len, s.plan.row_start, 6, mask=mask)
    assert torch.equal(y, x + B.forward(block.out, a.flatten(1)))
    path = torch.zeros(2, 3, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p)
    s.commit(path.cuda(), ints([3, 2]))
    plain = keys(x)[1]
    for b, p in enumerate(paths):
        for j, i in enumerate(p):
            row = 6 * b + i
            want = turn(plain[row:row + 1], ints([ctx[b] + j]))[0]
            assert torch.equal(cached(b, ctx[b] + j), want), (b, j)
    s.check()


def test_a_tree_is_not_turned_without_its_depths():
    s = V.random_stack(1, HIDDEN, HEADS, KV_HEADS, DIM, pages=8, page_size=PAGE, requests=1, width=4)
    x = torch.zeros(3, HIDDEN, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="depth"):
        s.step(x, ints([3]), 3, kv.ancestor_masks([-1, 0, 0]), rotate=Turner())
    with pytest.raises(ValueError, match="depth"):
        s.step(x, ints([3]), 3, kv.ancestor_masks([-1, 0, 0]), depth=ints([0, 1]), rotate=Turner())


def test_depths_refuse_what_is_no_tree():
    with pytest.raises(ValueError, match="parents"):
        kv.tree_depths([-1, 1])
    assert kv.tree_depths([]).tolist() == []
    chain = list(range(-1, 299))
    assert np.array_equal(kv.tree_depths(chain).cpu().numpy(), np.arange(300))
