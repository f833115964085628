"""Attention of drafted tokens over the paged cache against a plain 64-bit statement of it,
within what the kernel's roundings can add up to (kv_reference.attention_bounds)."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def tree_bits(rng, n):
    rows = []
    for i in range(n):
        p = int(rng.integers(-1, i)) if i else -1
        rows.append((1 << i) | (rows[p] if p >= 0 else 0))
    return rows


def words(rows, count):
    out = [[(r >> (64 * w)) & (2 ** 64 - 1) for w in range(count)] for r in rows]
    return [[x - 2 ** 64 if x >= 2 ** 63 else x for x in r] for r in out]


class Case:
    """Inputs of one call: random pages, q as a slice of a wider row, tree masks."""

    def __init__(self, ctx, new, heads, group, dim, page, dtype, mask="tree", heads_first=False,
                 seed=0, spare=3, mask_words=None, scale=None):
        rng = np.random.default_rng(seed)
        self.ctx, self.new, self.dim, self.page, self.dtype = ctx, new, dim, page, dtype
        self.scale = scale
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        width = max(need + [1]) + 1
        order = rng.permutation(sum(need) + spare)
        self.table = np.full((len(ctx), width), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = kv.KVCache.empty(len(order), page, heads, dim, dtype, heads_first=heads_first)
        mean = 2.0 * (rng.random((heads, dim)) < 0.05)
        for t, mu in ((self.cache.k, mean), (self.cache.v, 0.0)):
            t.copy_(torch.from_numpy((rng.standard_normal(t.shape) + mu).astype(np.float32)))
        rows, hq = sum(new), heads * group
        wide = torch.from_numpy(rng.standard_normal((rows, (hq + 2) * dim)).astype(np.float32))
        self.q = wide.to(dtype).cuda()[:, dim:-dim].unflatten(1, (hq, dim))
        self.start = ints(np.concatenate([[0], np.cumsum(new)]).tolist())
        self.max_new = max(new + [1])
        self.rows = None
        if mask == "tree":
            self.rows = [tree_bits(rng, n) for n in new]
        elif mask == "random":       # any bits at all, bits past the last token among them
            self.rows = [[int(rng.integers(0, 2 ** 62)) & int(rng.integers(0, 2 ** 62)) for _ in range(n)]
                         for n in new]
        elif mask == "none":
            self.rows = [[0] * n for n in new]
        count = mask_words or -(-self.max_new // 64)
        flat = [r for rows_ in self.rows for r in rows_] if self.rows is not None else []
        self.mask = None if self.rows is None else ints(words(flat, count), torch.int64).reshape(-1, count)

    def seen(self, b, i, j):
        return (self.rows[b][i] >> j) & 1 if self.rows is not None else j <= i

    def run(self, **kw):
        return kv.tree_attention(self.q, self.cache, ints(self.table.tolist()), ints(self.ctx),
                                 self.start, self.max_new, mask=self.mask, scale=self.scale,
                                 return_lse=True, **kw)

    def reference(self):
        f = [t.double().cpu().numpy() for t in (self.q, self.cache.k, self.cache.v)]
        scale = self.dim ** -0.5 if self.scale is None else self.scale
        ref, lse, weight = R.attention(*f, self.table.tolist(), self.page, self.ctx, self.new,
                                       self.seen, scale)
        keys = max(c + n for c, n in zip(self.ctx, self.new))
        fine = np.nan_to_num(f[1], nan=0.0, posinf=0.0, neginf=0.0)
        bounds = R.attention_bounds(f[0], fine, self.dim, keys, scale, self.dtype, ref, weight, lse)
        return ref, lse, bounds


def check(got, want):
    (out, lse), (ref, ref_lse, (of_out, of_lse)) = got, want
    B.tern_check()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(out), np.isnan(ref)) and np.array_equal(out[~fine & ~np.isnan(ref)],
                                                                           ref[~fine & ~np.isnan(ref)])
    assert (np.abs(out[fine] - ref[fine]) <= of_out[fine]).all()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    ok = np.isfinite(ref_lse)
    assert (np.abs(lse[ok] - ref_lse[ok]) <= of_lse[ok]).all()


CASES = [
    # ctx, new, heads, group, dim, page, dtype
    ([0], [1], 1, 1, 128, 16, BF),                       # a first token: sees itself alone
    ([1], [1], 1, 1, 64, 8, HF),
    ([0, 0], [5, 1], 2, 2, 64, 16, BF),
    ([63, 64, 65], [1, 1, 1], 2, 4, 128, 16, BF),        # around a tile's end
    ([127, 128, 129], [3, 2, 1], 1, 8, 128, 128, HF),
    ([700, 33, 250], [16, 1, 7], 5, 2, 128, 16, BF),
    ([300, 4], [64, 64], 2, 8, 128, 32, HF),             # 512 rows on each key head
    ([500], [130], 1, 3, 64, 64, BF),                    # three words of mask, odd group
    ([77], [256], 1, 2, 64, 16, HF),
    ([1000, 10, 300], [29, 3, 12], 2, 5, 256, 128, BF),
    ([257], [9], 3, 1, 256, 256, HF),
    ([2000] * 3, [1, 2, 1], 1, 16, 128, 8, BF),
    ([17, 0, 400], [4, 0, 4], 4, 4, 64, 16, BF),         # a request without new tokens
]


@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
@pytest.mark.parametrize("ctx,new,heads,group,dim,page,dtype", CASES)
def test_against_64_bits(ctx, new, heads, group, dim, page, dtype, mask):
    c = Case(ctx, new, heads, group, dim, page, dtype, mask=mask, seed=len(ctx) + new[0])
    check(c.run(), c.reference())


@pytest.mark.parametrize("group,new", [(1, 1), (4, 4), (8, 20)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_heads_of_rows_and_large_pages(dim, group, new):
    c = Case([333, 1025], [new, max(1, new - 1)], 2, group, dim, 256, BF, heads_first=True, seed=dim)
    check(c.run(), c.reference())


@pytest.mark.parametrize("dim,new", [(64, 3), (128, 40), (256, 17)])
def test_long_context_split_over_the_gpu(dim, new):
    """One request, one key head: its tiles are split over many CTAs and joined."""
    c = Case([20011], [new], 1, 2, dim, 16, BF, seed=new)
    check(c.run(), c.reference())


def test_many_requests():
    rng = np.random.default_rng(4)
    ctx, new = rng.integers(0, 200, 700).tolist(), rng.integers(0, 4, 700).tolist()
    c = Case(ctx, new, 1, 2, 64, 16, HF, seed=9)
    check(c.run(), c.reference())


@pytest.mark.parametrize("dim,new,group", [(64, 6, 2), (128, 33, 4), (256, 9, 1)])
def test_rows_that_see_nothing(dim, new, group):
    """No cached tokens and an empty mask: out 0, lse -infinity, beside rows that see some."""
    c = Case([0, 90], [new, new], 2, group, dim, 16, BF, mask="none")
    out, lse = c.run()
    assert (out[:new] == 0).all() and torch.isneginf(lse[:new]).all()
    check((out, lse), c.reference())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim,new,group", [(64, 6, 2), (128, 40, 4), (128, 3, 1), (256, 9, 4)])
def test_what_is_not_seen_has_no_influence(dim, new, group, value):
    """Everything past the last token, unused pages and the pages' ends, is not finite."""
    c = Case([50, 0, 129], [new, new, 1], 2, group, dim, 16, HF, seed=2)
    used = np.zeros((c.cache.pages, 16), dtype=bool)
    for b, (x, n) in enumerate(zip(c.ctx, c.new)):
        for p in range(x + n):
            used[c.table[b, p // 16], p % 16] = True
    want = c.reference()
    hole = torch.from_numpy(~used).cuda()
    c.cache.k[hole], c.cache.v[hole] = value, value
    check(c.run(), want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim,new,group", [(64, 6, 2), (128, 40, 4), (128, 3, 1), (256, 9, 4)])
def test_a_draft_that_is_not_finite_reaches_only_who_sees_it(dim, new, group, value):
    c = Case([50, 129], [new, 1], 2, group, dim, 16, HF, seed=3)
    want = c.reference()
    # token 1's values, and token 2's keys, of request 0
    at = [(c.table[0, (50 + i) // 16], (50 + i) % 16) for i in (1, 2)]
    c.cache.v[at[0][0], at[0][1], :, 5] = value
    c.cache.k[at[1][0], at[1][1], :, 7] = float("nan")
    out, lse = c.run()
    B.tern_check()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref, ref_lse, (of_out, of_lse) = want
    for row in range(sum(c.new)):
        first, second = (row < new and bool(c.seen(0, row, i)) for i in (1, 2))
        if second:
            assert np.isnan(out[row]).all() and np.isnan(lse[row]).all()
            continue
        assert (np.abs(lse[row] - ref_lse[row]) <= of_lse[row]).all()
        plain = np.ones(dim, dtype=bool)
        if first:
            plain[5] = False
            hit = out[row][:, 5]
            assert np.isnan(hit).all() if np.isnan(value) else (hit == value).all()
        assert (np.abs(out[row] - ref[row])[:, plain] <= of_out[row][:, plain]).all()


def test_cached_keys_that_are_not_finite_reach_every_row():
    c = Case([100], [5], 1, 2, 128, 16, BF)
    c.cache.k[c.table[0, 2], 3] = float("nan")
    out, lse = c.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("group", [3, 5, 7, 12, 130])
def test_groups_that_do_not_divide_a_tile(group):
    c = Case([150, 9], [31, 12] if group < 100 else [2, 1], 2, group, 64, 32, BF, seed=group)
    check(c.run(), c.reference())


@pytest.mark.parametrize("dim,new", [(64, 60), (128, 11), (128, 40), (256, 12)])
def test_negative_scale(dim, new):
    c = Case([300, 70], [new, 2], 2, 4, dim, 16, HF, scale=-0.15, seed=dim)
    check(c.run(), c.reference())


def test_scores_far_apart_and_negative_scale():
    c = Case([600, 40], [7, 3], 2, 2, 128, 16, BF, scale=3.0)
    check(c.run(), c.reference())
    c = Case([600, 40], [7, 3], 2, 2, 64, 16, HF, scale=-0.2)
    check(c.run(), c.reference())


def test_more_mask_words_than_needed_and_the_callers_buffers():
    c = Case([100, 31], [5, 60], 2, 2, 128, 16, BF, mask_words=4)
    out = poison(torch.empty((65, 4, 128), dtype=BF, device="cuda"))
    lse = poison(torch.empty((65, 4), dtype=torch.float32, device="cuda"))
    ws = B.Workspace()
    for _ in range(2):
        got = c.run(out=out, lse=lse, ws=ws)
        assert got[0] is out and got[1] is lse
        check(got, c.reference())


def test_table_entries_out_of_range_are_zero_keys():
    """A page that does not exist is not followed: its keys and values count as zero."""
    c = Case([40], [2], 1, 2, 64, 16, BF)
    zero = next(p for p in range(c.cache.pages) if p not in c.table)
    c.cache.k[zero], c.cache.v[zero] = 0, 0
    c.table[0, 1] = zero
    want = c.reference()
    for bad in (-1, c.cache.pages, 2 ** 31 - 1, -2 ** 31):
        c.table[0, 1] = bad
        check(c.run(), want)


def test_same_bits_again_and_on_another_stream():
    c = Case([3000, 129, 7], [9, 16, 1], 2, 4, 128, 16, BF)
    first = c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for kw in ({}, {"stream": side}, {"stream": side.cuda_stream}):
        again = c.run(**kw)
        torch.cuda.synchronize()
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(first[1], again[1])


def test_captured_and_replayed_with_other_lengths():
    c = Case([200, 900], [4, 4], 2, 2, 128, 16, BF)
    table, ctx, ws = ints(c.table.tolist()), ints([3, 1]), B.Workspace()
    out = torch.empty((8, 4, 128), dtype=BF, device="cuda")
    lse = torch.empty((8, 4), dtype=torch.float32, device="cuda")

    def call():
        kv.tree_attention(c.q, c.cache, table, ctx, c.start, 4, mask=c.mask, out=out, lse=lse, ws=ws,
                          return_lse=True)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    ctx.copy_(ints(c.ctx))
    graph.replay()
    check((out, lse), c.reference())


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, the request on its first and last pages."""
    pages, page, heads, dim = 2 ** 32 // (64 * 4 * 128) + 9, 64, 4, 128
    cache = kv.KVCache.empty(pages, page, heads, dim)
    table = [[pages - 1, 0, pages - 2]]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for pg in table[0]:
        cache.k[pg] = torch.randn(page, heads, dim, device="cuda", generator=gen).to(BF)
        cache.v[pg] = torch.randn(page, heads, dim, device="cuda", generator=gen).to(BF)
    ctx, n = 160, 5
    new = torch.randn(n, heads, dim, device="cuda", generator=gen).to(BF)
    plan = kv.kv_plan(ints([ctx]), ints([n]), ints(table), ints([], torch.int32), page, n)
    kv.kv_write(cache, new, -new, plan.slots)
    q = torch.randn(n, 2 * heads, dim, device="cuda", generator=gen).to(BF)
    got = kv.tree_attention(q, cache, ints(table), ints([ctx]), plan.row_start, n, return_lse=True)
    B.tern_check()
    k = cache.k[table[0]].double().cpu().numpy()
    v = cache.v[table[0]].double().cpu().numpy()
    assert np.array_equal(k.reshape(-1, heads, dim)[ctx:ctx + n], new.double().cpu().numpy())
    qf = q.double().cpu().numpy()
    ref, lse, weight = R.attention(qf, k, v, [[0, 1, 2]], page, [ctx], [n], lambda b, i, j: j <= i,
                                   dim ** -0.5)
    bounds = R.attention_bounds(qf, k, dim, ctx + n, dim ** -0.5, BF, ref, weight, lse)
    check(got, (ref, lse, bounds))
