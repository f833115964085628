"""A step of speculative decoding through ternary blocks: the four cache calls together, as a
server makes them, with lengths that only the GPU knows."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from ternary_weight_linear_block_gb300 import verify as V
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_verification_steps():
    requests, hidden, heads, kv_heads, dim, page = 3, 1024, 16, 4, 64, 16
    s = V.random_stack(2, hidden, heads, kv_heads, dim, pages=40, page_size=page, requests=requests,
                       width=12, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def states(rows):
        return torch.randn(rows, hidden, generator=gen, device="cuda").to(torch.bfloat16)

    prompt = [33, 7, 70]
    s.step(states(sum(prompt)), ints(prompt), max(prompt))
    s.commit(ints([list(range(70))] * requests), ints(prompt))
    assert s.ctx_len.tolist() == prompt
    taken = [-(-p // page) for p in prompt]
    ctx, accepted = prompt, [[0, 2, 4], [0], [0, 1, 3]]
    trees = [[-1, 0, 0, 1, 2], [-1, 0, 1, 2, 3], [-1, 0, 0, 1, 1]]
    mask = torch.cat([kv.ancestor_masks(t) for t in trees])
    for _ in range(4):
        x, new = states(15), [5, 5, 5]
        y = s.step(x, ints(new), 5, mask)
        B.tern_check()
        assert torch.isfinite(y).all()
        # every table entry in use is a page of its own
        table = s.table.tolist()
        used = [p for b in range(requests) for p in table[b][:-(-(ctx[b] + 5) // page)]]
        assert len(set(used)) == len(used) and min(used) >= 0
        # pages of drafts that were not kept are used again: none are taken twice
        taken = [max(h, -(-(c + 5) // page)) for h, c in zip(taken, ctx)]
        assert s.held.tolist() == taken and s.free_head.tolist() == [sum(taken)]
        # the first block's attention against its 64-bit statement
        block = s.blocks[0]
        qkv = B.forward(block.qkv, x, ws=s.ws_linear)
        q = qkv[:, :heads * dim].unflatten(1, (heads, dim))
        k = qkv[:, heads * dim:(heads + kv_heads) * dim].unflatten(1, (kv_heads, dim))
        got = kv.tree_attention(q, block.cache, s.table, s.ctx_len, s.plan.row_start, 5, mask=mask)
        f = [t.double().cpu().numpy() for t in (q, block.cache.k, block.cache.v)]
        bits = mask[:, 0].tolist()
        ref, lse, weight = R.attention(*f, table, page, ctx, new, lambda b, i, j: (bits[5 * b + i] >> j) & 1,
                                       dim ** -0.5)
        seen = np.nan_to_num(f[1][sorted(set(used))])
        bounds, _ = R.attention_bounds(f[0], seen, dim, max(ctx) + 5, dim ** -0.5, torch.bfloat16, ref,
                                       weight, lse)
        assert (np.abs(got.double().cpu().numpy() - ref) <= bounds).all()
        # the accepted tokens' keys move to the end of the context, in both blocks
        before = [b.cache.k.clone() for b in s.blocks]
        path = torch.zeros((requests, 3), dtype=torch.int32)
        for b, p in enumerate(accepted):
            path[b, :len(p)] = torch.tensor(p)
        s.commit(path.cuda(), ints([len(p) for p in accepted]))
        for old, blk in zip(before, s.blocks):
            for b, p in enumerate(accepted):
                for j, i in enumerate(p):
                    a, z = ctx[b] + i, ctx[b] + j
                    assert torch.equal(blk.cache.k[table[b][z // page], z % page],
                                       old[table[b][a // page], a % page])
        assert torch.equal(before[0][s.plan.slots // page, s.plan.slots % page], k)
        ctx = [c + len(p) for c, p in zip(ctx, accepted)]
        assert s.ctx_len.tolist() == ctx


def test_blocks_that_do_not_fit():
    s = V.random_stack(1, 1024, 16, 4, 64, pages=4, page_size=16, requests=1, width=2)
    b = s.blocks[0]
    with pytest.raises(ValueError):
        V.Block(b.out, b.qkv, b.cache)
