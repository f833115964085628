"""The tile kernel's steady state: long runs of tiles of one item in a CTA, many items one after
another, and row maxima that keep moving, against the definition in 64 bits."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
PAGE = 64
# head size, query heads on a key head, drafts: 48, 32, 320 and 40 rows (320: two streams, else one accumulator)
FORMS = [(64, 8, 6), (128, 4, 8), (128, 8, 40), (256, 8, 5)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Run:
    """Requests of ``ctx`` cached tokens and a tree of drafts each; ``rise``: what a row's scores
    gain (base 2) every ``every`` keys, falling for every third token."""

    def __init__(self, ctx, new, heads, group, dim, dtype, seed, rise=0.0, every=300):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.new, self.heads, self.group, self.dim, self.dtype = ctx, new, heads, group, dim, dtype
        need = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
        order = rng.permutation(sum(need))
        self.table = np.full((len(ctx), max(need)), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = kv.KVCache.empty(len(order), PAGE, heads, dim, dtype)
        for t in (self.cache.k, self.cache.v):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.q = torch.randn((sum(new), heads * group, dim), generator=gen, device="cuda").to(dtype)
        if rise:
            self.q[:, :, 0] = 4.0
            self.q[::3, :, 0] = -4.0
            step = rise / (4 * dim ** -0.5 * np.log2(np.e))
            for b, n in enumerate(need):
                j = torch.arange(n * PAGE, device="cuda") // every
                # up for a while, then from far below again
                self.cache.k[self.table[b, :n].tolist(), :, :, 0] = \
                    ((j % 17).to(torch.float32) * step).to(dtype).reshape(n, PAGE, 1).expand(-1, -1, heads)
        rows = []
        for n in new:
            own = []
            for i in range(n):
                p = int(rng.integers(max(-1, i - 5), i)) if i else -1
                own.append((1 << i) | (own[p] if p >= 0 else 0))
            rows.append(own)
        self.rows = rows
        words = [w - 2 ** 64 if w >= 2 ** 63 else w for r in rows for w in r]
        self.mask = torch.tensor(words, dtype=torch.int64, device="cuda").reshape(-1, 1)

    def call(self):
        return kv.tree_attention(self.q, self.cache, ints(self.table.tolist()), ints(self.ctx),
                                 ints(self.start.tolist()), max(self.new), mask=self.mask, return_lse=True)

    def check(self, got, bad=()):
        """``bad``: requests whose draft 1 has an infinite value in column 5 of head 0."""
        B.tern_check()
        out, lse = got
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            used = self.table[b, :-(-(c + n) // PAGE)].tolist()
            lo, hi = self.start[b], self.start[b + 1]
            seen = torch.ones(n, 1, c + n, dtype=torch.bool, device="cuda")
            for i, word in enumerate(self.rows[b]):
                seen[i, 0, c:] = torch.tensor([(word >> j) & 1 for j in range(n)], dtype=torch.bool)
            for h in range(self.heads):
                k = self.cache.k[used, :, h].flatten(0, 1)[:c + n].double()
                v = self.cache.v[used, :, h].flatten(0, 1)[:c + n].double()
                q = self.q[lo:hi, h * self.group:(h + 1) * self.group].double()
                s = (q @ k.T * self.dim ** -0.5).masked_fill(~seen, float("-inf"))
                p = s.softmax(-1)
                hit = b in bad and h == 0
                if hit:
                    v[c + 1, 5] = 0
                ref, weight = (p @ v).cpu().numpy(), (p @ v.abs()).cpu().numpy()
                ref_lse = s.logsumexp(-1).cpu().numpy()
                norms = [np.full((1, 1), float(x.norm(dim=-1).max())) for x in (q, k)]
                of_out, of_lse = R.attention_bounds(*norms, self.dim, c + n, self.dim ** -0.5, self.dtype, ref,
                                                    weight, ref_lse)
                mine = out[lo:hi, h * self.group:(h + 1) * self.group].double().cpu().numpy()
                if hit:
                    who = np.array([(w >> 1) & 1 for w in self.rows[b]], dtype=bool)
                    assert np.isposinf(mine[who, :, 5]).all()
                    mine[who, :, 5] = ref[who, :, 5]
                assert (np.abs(mine - ref) <= of_out).all(), (b, h)
                l = lse[lo:hi, h * self.group:(h + 1) * self.group].double().cpu().numpy()
                assert (np.abs(l - ref_lse) <= of_lse).all(), (b, h)


@pytest.mark.parametrize("rise", [0.0, 3.0, 12.0])
@pytest.mark.parametrize("dim,group,new", FORMS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_long_items(dtype, dim, group, new, rise):
    """About ten tiles and more of one item for each of the GPU's CTAs."""
    tile = 64 if dim == 256 else 128
    rows = 1 + (new * group > 256)
    ctx = 152 * 11 * tile // (2 * rows)
    c = Run([ctx + 37, ctx], [new, new - 1], 1, group, dim, dtype, seed=dim + new, rise=rise)
    first = c.call()
    c.check(first)
    again = c.call()
    assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("rise", [0.0, 12.0])
@pytest.mark.parametrize("dim,group,new", FORMS)
def test_hundreds_of_short_items(dim, group, new, rise):
    """Four items and more for each CTA, of which some have a draft that is not finite."""
    rng = np.random.default_rng(dim)
    requests = 320
    ctx = rng.integers(0, 700, requests).tolist()
    tokens = rng.integers(2, new + 1, requests).tolist()
    tokens[5] = new
    c = Run(ctx, tokens, 2, group, dim, HF, seed=new, rise=rise, every=90)
    bad = list(range(3, requests, 7))
    for b in bad:
        at = ctx[b] + 1
        c.cache.v[c.table[b, at // PAGE], at % PAGE, 0, 5] = float("inf")
    c.check(c.call(), bad)


@pytest.mark.parametrize("dim,group,new", FORMS)
def test_one_long_item_among_short_ones(dim, group, new):
    ctx = [int(x) for x in np.random.default_rng(7).integers(0, 300, 200)]
    ctx[100] = 90000
    c = Run(ctx, [new] * 200, 1, group, dim, BF, seed=3, rise=9.0)
    c.check(c.call())
