"""Verification of drafted-token trees through attention blocks of ternary linears.

``VerifyStack`` runs one step of speculative decoding over a stack of blocks
(qkv linear, paged attention, output linear): the step's pages and slots are
planned on the GPU, every block writes its new keys and values (turned by the
caller's rotary embedding, if it gives one) and attends over the cache, and once the caller knows the accepted paths, ``commit``
makes them contiguous in all blocks at once.  ``accept`` finds the accepted
paths from the tokens that were sampled (sampling.sample) and commits them.
Caches are of 16 or 8 bits.  The norms around a block and the MLP belong to
the model around it; here a block's output is added to its input.

``python -m ternary_weight_linear_block_gb300.verify`` runs a small stack of
random weights over 8-bit caches: a prompt, then steps that verify a tree for
each request with sampled tokens.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B
from . import kv
from . import sampling

MAX_NEW = 256      # new tokens of a request in one step, as tern_tree_attention takes them


_FLAGS = {1: "the cache has no free pages left", 2: "a request is longer than its table row's pages",
          4: "new_len has more rows than x", 8: "a negative length"}


@dataclass
class Block:
    """One attention block: qkv [(heads + 2 kv_heads) dim, hidden] and output
    [hidden, heads dim] ternary layers, its cache, and the weights [dim] of the
    norms of every head's queries and keys, if it has them."""
    qkv: B.PackedLayer
    out: B.PackedLayer
    cache: kv.KVCache | kv.KVCache8
    q_norm: torch.Tensor | None = None
    k_norm: torch.Tensor | None = None
    eps: float = 1e-6

    def __post_init__(self):
        self.heads = self.out.k // self.cache.dim
        if self.qkv.n != (self.heads + 2 * self.cache.heads) * self.cache.dim or \
                self.out.k != self.heads * self.cache.dim or self.qkv.k != self.out.n:
            raise ValueError("qkv, out: sizes do not belong together")


class VerifyStack:
    """Blocks that share block tables and lengths.  ``table`` int32 [requests,
    width] and ``ctx_len`` int32 [requests] start empty; pages come from the
    cache's own, in order, and stay with their request."""

    def __init__(self, blocks: list[Block], requests: int, width: int):
        self.blocks = blocks
        cache = blocks[0].cache
        dev = cache.device
        self.requests, self.page_size = requests, cache.page_size
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=dev)
        self.ctx_len = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.free_pages = torch.arange(cache.pages, dtype=torch.int32, device=dev)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=dev)
        # pages in each table row, of this step and the next
        self.held, self.held_next = (torch.zeros(requests, dtype=torch.int32, device=dev)
                                     for _ in range(2))
        # the linears' and the attention's workspaces: the attention leaves
        # partial sums behind, which the linears would have to zero again
        self.ws_linear, self.ws_attention = B.Workspace(dev), B.Workspace(dev)
        self.plan = None

    def step(self, x: torch.Tensor, new_len: torch.Tensor, max_new: int,
             mask: torch.Tensor | None = None, depth: torch.Tensor | None = None,
             rotate=None, positions: torch.Tensor | None = None) -> torch.Tensor:
        """Hidden states [rows, hidden] of the new tokens through all blocks;
        new_len int32 [requests] rows each (``max_new`` at most, which is 256
        at most: a longer prompt goes in parts), masked as
        kv.tree_attention's ``mask``.  The tokens stay drafts until commit.
        Whether they all had a place, only ``check`` says.

        ``rotate`` is a kv.Rotary, which turns every block's queries and keys as
        they are written (kv.rotate_write, with the block's norms), or a function:
        ``rotate(q, k, positions)`` returns the queries [rows, heads, dim] and
        keys [rows, kv_heads, dim] with their position in them; positions are
        int32 [rows].  With a mask, ``depth`` (kv.tree_depths of each request's
        tree, int32 [rows]) says where the tokens stand; without one they are
        chains.  ``positions`` gives other ones, int32 [rows], or [axes, rows]
        for a kv.Rotary of several axes."""
        rows = x.shape[0]
        fused = rotate is None or isinstance(rotate, kv.Rotary)
        if not fused and any(b.q_norm is not None or b.k_norm is not None for b in self.blocks):
            raise ValueError("rotate: expected a kv.Rotary, as the blocks have norms of queries or keys")
        if positions is not None and (rotate is None or positions.shape[-1] != rows):
            raise ValueError("positions: expected rotate, and one of every row")
        if max_new > MAX_NEW:
            raise ValueError(f"max_new: expected {MAX_NEW} at most, longer prompts in parts")
        if rotate is not None and mask is not None and positions is None and (depth is None or depth.shape != (rows,)):
            raise ValueError("depth: expected the depth of every row's token, as mask describes a tree")
        self.plan = kv.kv_plan(self.ctx_len, new_len, self.table, self.free_pages, self.page_size,
                               rows, free_head=self.free_head, held=self.held,
                               held_out=self.held_next)
        at = positions
        if rotate is not None and positions is None:
            at = self.plan.positions
            if depth is not None:
                at = self.ctx_len[self.plan.request.clamp(min=0)] + depth
        for block in self.blocks:
            x = x + self.block(block, x, max_new, mask,
                               None if fused else (lambda q, k: rotate(q, k, at)),
                               rotate if fused else None, at)
        # only now, so that after a call that was refused the next step plans
        # with the same pages
        self.held, self.held_next = self.held_next, self.held
        self.free_head = self.plan.info[2:3]
        return x

    def check(self):
        """Raises if the last step's tokens did not all fit, or if a wait on
        the GPU gave up (synchronises).  A token without a page is not
        written, the step's other rows see it as a zero key, and commit cuts
        a path there."""
        B.tern_check()
        flags = int(self.plan.info[3])
        what = [name for bit, name in _FLAGS.items() if flags & bit]
        if what:
            raise RuntimeError("step: " + ", ".join(what))

    def block(self, block: Block, x: torch.Tensor, max_new: int, mask, rotate=None,
              rotary: kv.Rotary | None = None, positions: torch.Tensor | None = None) -> torch.Tensor:
        cache, p = block.cache, self.plan
        qkv = B.forward(block.qkv, x, ws=self.ws_linear)
        q, k, v = (t.unflatten(1, (-1, cache.dim)) for t in qkv.split(
            [block.heads * cache.dim, cache.heads * cache.dim, cache.heads * cache.dim], dim=1))
        if rotate is not None:
            q, k = rotate(q, k)
        if rotary is None and block.q_norm is None and block.k_norm is None:
            kv.kv_write(cache, k, v, p.slots)
        else:
            q = kv.rotate_write(cache, q, k, v, p.slots, rotary, positions, block.q_norm, block.k_norm, block.eps)
        a = kv.tree_attention(q, cache, self.table, self.ctx_len, p.row_start, max_new, mask=mask,
                              ws=self.ws_attention)
        return B.forward(block.out, a.flatten(1), ws=self.ws_linear)

    def commit(self, path: torch.Tensor, path_len: torch.Tensor) -> torch.Tensor:
        """Keep the accepted path of every request (kv.kv_commit), in all
        blocks; returns the new lengths."""
        self.ctx_len = kv.kv_commit([b.cache for b in self.blocks], self.table, self.ctx_len, path,
                                    path_len)
        return self.ctx_len


    def accept(self, tokens: torch.Tensor, target: torch.Tensor, parents: torch.Tensor,
               max_new: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """Commit the path of every request's tree that the sampled tokens
        agree with (sampling.accept, of the last step's rows); returns it: path,
        path_len and the requests' next tokens."""
        path, path_len, following = sampling.accept(tokens, target, parents, self.plan.row_start, max_new)
        self.commit(path, path_len)
        return path, path_len, following


def random_stack(layers: int, hidden: int, heads: int, kv_heads: int, dim: int, pages: int,
                 page_size: int, requests: int, width: int, seed: int = 0,
                 device="cuda", cache=torch.bfloat16, norms: bool = False) -> VerifyStack:
    """A stack of random ternary blocks (for examples and tests); ``cache`` is
    the type that it holds, of 16 or 8 bits."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def linear(n, k):
        codes = torch.randint(-1, 2, (n, k), generator=gen, device=device, dtype=torch.int8)
        scales = (0.02 * torch.rand(n, k // 128, generator=gen, device=device) + 0.005).half()
        return B.pack_layer(codes, scales)

    kind = kv.KVCache if cache in (torch.bfloat16, torch.float16) else kv.KVCache8

    def norm():
        return (1 + 0.1 * torch.randn(dim, generator=gen, device=device)).to(torch.bfloat16) if norms else None

    return VerifyStack([Block(linear((heads + 2 * kv_heads) * dim, hidden), linear(hidden, heads * dim),
                              kind.empty(pages, page_size, kv_heads, dim, cache, device), norm(), norm())
                        for _ in range(layers)], requests, width)


def rotary(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, base: float = 1e6):
    """A rotary embedding as VerifyStack.step's ``rotate`` (for the example; plain torch)."""
    half = q.shape[-1] // 2
    rate = base ** (-torch.arange(half, device=q.device) / half)
    angle = positions[:, None, None] * rate
    cos, sin = angle.cos(), angle.sin()

    def turn(x):
        a, b = x.float().chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(x.dtype)
    return turn(q), turn(k)


def main():
    requests, hidden, vocab, tree = 2, 5120, 32768, [-1, 0, 0, 1, 1, 2, 3]
    stack = random_stack(layers=2, hidden=hidden, heads=40, kv_heads=20, dim=128, pages=64, page_size=16,
                         requests=requests, width=32, cache=torch.int8, norms=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    head = B.pack_layer(torch.randint(-1, 2, (vocab, hidden), generator=gen, device="cuda", dtype=torch.int8),
                        (1e-3 * torch.rand(vocab, hidden // 128, generator=gen, device="cuda") + 1e-4).half())
    turn = kv.Rotary.geometric(128)

    def states(rows):
        return torch.randn(rows, hidden, generator=gen, device="cuda").to(torch.bfloat16)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def sampled(y, temperature):
        u = torch.rand(y.shape[0], generator=gen, device="cuda")
        return sampling.sample(B.forward(head, y), u, temperature=torch.full_like(u, temperature),
                               top_p=torch.full_like(u, 0.9))

    prompt = [100, 37]                                   # a prompt is a chain whose tokens all stay
    stack.step(states(sum(prompt)), ints(prompt), max(prompt), rotate=turn)
    stack.commit(ints([list(range(max(prompt)))] * requests), ints(prompt))
    mask, depth = kv.ancestor_masks(tree).repeat(requests, 1), kv.tree_depths(tree).repeat(requests)
    parents = ints(tree * requests)
    for temperature in 0.0, 1.0:
        y = stack.step(states(requests * len(tree)), ints([len(tree)] * requests), len(tree), mask, depth, turn)
        target = sampled(y, temperature)
        # drafts as a draft model might have made them: the first child of every token is right
        tokens = torch.full_like(target, -1)
        for b in range(requests):
            for i in range(1, len(tree)):
                tokens[b * len(tree) + i] = target[b * len(tree) + tree[i]] if i in (1, 3, 5) else -1
        _, kept, following = stack.accept(tokens, target, parents, len(tree))
        stack.check()
        print(f"verified {tuple(y.shape)} drafts, kept {kept.tolist()}, next {following.tolist()}, "
              f"lengths now {stack.ctx_len.tolist()}, finite: {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
