"""A whole step over 8-bit caches: rows rotated as they are written, attention, sampling,
acceptance and commit, as a server makes them, and captured in one graph."""

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from ternary_weight_linear_block_gb300 import sampling
from ternary_weight_linear_block_gb300 import verify as V
from tests import kv8_reference as R8
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
HIDDEN, HEADS, KV_HEADS, DIM, VOCAB = 1024, 16, 4, 64, 2048
TREE = [-1, 0, 0, 1, 2]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(cache, seed=3, norms=True):
    return V.random_stack(2, HIDDEN, HEADS, KV_HEADS, DIM, pages=40, page_size=16, requests=3, width=12, seed=seed,
                          cache=cache, norms=norms)


def random_head(gen):
    codes = torch.randint(-1, 2, (VOCAB, HIDDEN), generator=gen, device="cuda", dtype=torch.int8)
    return B.pack_layer(codes, (2e-3 * torch.rand(VOCAB, HIDDEN // 128, generator=gen, device="cuda") + 1e-4).half())


def states(gen, rows):
    return torch.randn(rows, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16)


def fill(stack, gen, turn, prompt=(33, 7, 70)):
    stack.step(states(gen, sum(prompt)), ints(prompt), max(prompt), rotate=turn)
    stack.commit(ints([list(range(max(prompt)))] * 3), ints(prompt))


@pytest.mark.parametrize("cache", [torch.int8, torch.float8_e4m3fn, torch.bfloat16])
def test_steps(cache):
    """Lengths, kept drafts and next tokens as the plain statement has them; and the caches of 8 bits give
    what those of 16 do, to the codes' rounding."""
    stack, plain = make(cache), make(torch.bfloat16)
    turn, gen = kv.Rotary.geometric(DIM), torch.Generator(device="cuda").manual_seed(5)
    head = random_head(gen)
    at = gen.get_state()
    fill(stack, gen, turn)
    gen.set_state(at)
    fill(plain, gen, turn)
    mask, depth = kv.ancestor_masks(TREE).repeat(3, 1), kv.tree_depths(TREE).repeat(3)
    ctx = [33, 7, 70]
    for step in range(3):
        x = states(gen, 15)
        y = stack.step(x, ints([5] * 3), 5, mask, depth, turn)
        want = plain.step(x, ints([5] * 3), 5, mask, depth, turn)
        assert float((y.float() - want.float()).norm() / want.float().norm()) < 0.05
        u = torch.rand(15, generator=gen, device="cuda")
        target = sampling.sample(B.forward(head, y), u, top_p=torch.full_like(u, 0.9))
        tokens = torch.randint(VOCAB, (15,), generator=gen, device="cuda", dtype=torch.int32)
        tokens[1], tokens[3], tokens[5 + 2] = target[0], target[1], target[5]
        path, kept, following = stack.accept(tokens, target, ints(TREE * 3), 5)
        ref = R8.accept(tokens.tolist(), target.tolist(), TREE * 3, [0, 5, 10, 15], 5)
        assert (path.tolist(), kept.tolist(), following.tolist()) == tuple(ref)
        assert ref[1][0] >= 3 and ref[1][1] >= 2
        plain.commit(path, kept)
        ctx = [c + n for c, n in zip(ctx, ref[1])]
        assert stack.ctx_len.tolist() == ctx
        stack.check()


def test_a_step_in_one_graph():
    """Captured once, replayed as states, drafts and lengths change: the same as the calls one by one."""
    turn, gen = kv.Rotary.geometric(DIM), torch.Generator(device="cuda").manual_seed(7)
    head = random_head(gen)
    mask, depth, parents = (kv.ancestor_masks(TREE).repeat(3, 1), kv.tree_depths(TREE).repeat(3), ints(TREE * 3))
    new = ints([5] * 3)
    s = make(torch.int8)
    fill(s, gen, turn)
    x, u, tokens = states(gen, 15), torch.rand(15, generator=gen, device="cuda"), ints([0] * 15)
    low = torch.full_like(u, 0.8)

    def step():
        y = s.step(x, new, 5, mask, depth, turn)
        target = sampling.sample(B.forward(head, y, ws=s.ws_linear), u, temperature=low, top_p=low)
        path, kept, following = sampling.accept(tokens, target, parents, s.plan.row_start, 5)
        out = kv.kv_commit([b.cache for b in s.blocks], s.table, s.ctx_len, path, kept)
        return y, target, path, kept, following, out

    held, head_at = s.held.clone(), s.free_head.clone()
    first = [t.clone() for t in step()]                 # (also makes the workspaces)
    s.held.copy_(held), s.free_head.copy_(head_at)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    s.held, s.free_head = held, head_at
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first))
    # other states, random numbers and drafts; the lengths go on on the GPU
    for _ in range(3):
        s.ctx_len.copy_(out[-1])
        x.copy_(states(gen, 15))
        u.copy_(torch.rand(15, generator=gen, device="cuda"))
        tokens.copy_(out[1].roll(1))
        before = s.ctx_len.tolist()
        graph.replay()
        torch.cuda.synchronize()
        B.tern_check()
        ref = R8.accept(tokens.tolist(), out[1].tolist(), TREE * 3, [0, 5, 10, 15], 5)
        assert (out[2].tolist(), out[3].tolist(), out[4].tolist()) == tuple(ref)
        assert out[-1].tolist() == [c + n for c, n in zip(before, ref[1])]


def test_several_axes_and_norms_only():
    """Positions of a caller's own, and blocks with norms and no rotation."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    s = make(torch.int8)
    turn = kv.Rotary([1e4 ** (-j / 32) for j in range(32)], axis=[j % 3 for j in range(32)])
    where = torch.stack([torch.arange(12), torch.arange(12) // 4, torch.arange(12) % 4]).int().cuda()
    y = s.step(states(gen, 12), ints([4] * 3), 4, rotate=turn, positions=where)
    assert torch.isfinite(y).all()
    s.check()
    y = make(torch.bfloat16).step(states(gen, 12), ints([4] * 3), 4)
    assert torch.isfinite(y).all()


def test_refusals():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = states(gen, 3)
    with pytest.raises(ValueError, match="kv.Rotary"):
        make(torch.int8).step(x, ints([1] * 3), 1, rotate=V.rotary)
    with pytest.raises(ValueError, match="positions"):
        make(torch.int8).step(x, ints([1] * 3), 1, positions=ints([0, 0, 0]))
    with pytest.raises(ValueError, match="positions"):
        make(torch.int8).step(x, ints([1] * 3), 1, rotate=kv.Rotary.geometric(64), positions=ints([0, 0]))
    with pytest.raises(ValueError, match="depth"):
        make(torch.int8).step(x, ints([1] * 3), 1, kv.ancestor_masks([-1] * 3), rotate=kv.Rotary.geometric(64))
