"""The paged cache's plan, write and commit against plain statements of them: whole numbers
and copied rows, so every comparison is exact."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import kv
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def make_plan_case(rng, requests, ctx, new, page, spare=0, short=0):
    c = rng.integers(0, ctx + 1, requests).tolist()
    n = rng.integers(0, new + 1, requests).tolist()
    held = [-(-x // page) for x in c]
    width = max([-(-(x + y) // page) for x, y in zip(c, n)] + [1]) + spare
    need = sum(-(-(x + y) // page) - h for x, y, h in zip(c, n, held))
    order = rng.permutation(sum(held) + need + 5)
    table, at = np.full((requests, width), -7), 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    return c, n, table.tolist(), order[at:len(order) - short].tolist()


def check_plan(c, n, page, table, free, head, capacity, buffers=False):
    want = R.plan(c, n, page, table, free, head, capacity)
    t = ints(table).reshape(len(c), -1)
    plan = None
    if buffers:
        plan = kv.KVPlan.empty(len(c), capacity)
        for x in plan:
            poison(x)
    got = kv.kv_plan(ints(c), ints(n), t, ints(free), page, capacity,
                     free_head=ints([head]) if head else None, plan=plan)
    assert t.tolist() == want[0]
    for name, w in zip(("row_start", "slots", "positions", "request", "info"), want[1:]):
        assert getattr(got, name).tolist() == w, name


@pytest.mark.parametrize("requests,ctx,new,page", [
    (1, 0, 1, 16), (1, 100, 17, 16), (3, 64, 0, 16), (16, 5000, 16, 16), (7, 40, 33, 8),
    (511, 30, 5, 32), (512, 30, 5, 1), (513, 30, 5, 64), (1100, 9, 3, 2), (2, 10, 5000, 128),
    (5, 3, 1, 65536)])
def test_plan(requests, ctx, new, page):
    rng = np.random.default_rng(requests * 131 + new)
    c, n, table, free = make_plan_case(rng, requests, ctx, new, page, spare=2)
    check_plan(c, n, page, table, free, 0, sum(n))
    check_plan(c, n, page, table, [0, 0, 0] + free, 3, sum(n) + 9, buffers=True)


def test_plan_what_does_not_fit():
    rng = np.random.default_rng(3)
    c, n, table, free = make_plan_case(rng, 9, 50, 40, 16, short=9)
    check_plan(c, n, 16, table, free, 0, sum(n))               # the free pages run out
    check_plan(c, n, 16, table, [], 0, sum(n))
    check_plan(c, n, 16, [r[:2] for r in table], free, 0, sum(n))   # table rows too short
    check_plan(c, n, 16, table, free, 0, sum(n) - 5)           # fewer rows planned than asked
    check_plan(c, n, 16, table, free, 0, 0)
    check_plan([-3, 7, 20], [4, -1, 3], 16, [[5, 6], [1, 2], [3, 4]], [8, 9], 0, 8)


def test_plan_of_no_requests():
    got = kv.kv_plan(ints([]), ints([]), ints([]).reshape(0, 4), ints([1, 2]), 16, 3)
    assert got.row_start.tolist() == [0] and got.slots.tolist() == [-1] * 3
    assert got.info.tolist() == [0, 0, 0, 0]


def test_plan_with_pages_held_from_a_step_before():
    """A request that kept few of its drafts has pages to spare; one has fewer than its tokens."""
    table = torch.tensor([[3, 4, 5, -1], [6, -1, -1, -1], [7, 8, -1, -1]], dtype=torch.int32, device="cuda")
    held, out = ints([3, 1, 2]), poison(torch.empty(3, dtype=torch.int32, device="cuda"))
    got = kv.kv_plan(ints([18, 16, 33]), ints([9, 1, 2]), table, ints([20, 21, 22]), 16, 12, held=held,
                     held_out=out)
    assert table.tolist() == [[3, 4, 5, -1], [6, 20, -1, -1], [7, 8, 21, -1]]
    assert out.tolist() == [3, 2, 3] and got.info.tolist() == [12, 2, 2, 0]
    want = [4 * 16 + i for i in range(2, 11)] + [20 * 16] + [21 * 16 + 1, 21 * 16 + 2]
    assert got.slots.tolist() == want


def test_plan_is_the_next_steps_free_head():
    free = ints([9, 8, 7, 6, 5])
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    first = kv.kv_plan(ints([0, 0]), ints([17, 3]), table, free, 16, 20)
    second = kv.kv_plan(ints([17, 3]), ints([1, 20]), table, free, 16, 21, free_head=first.info[2:3])
    assert table.tolist() == [[9, 8, -1, -1], [7, 6, -1, -1]]
    assert second.info.tolist() == [21, 1, 4, 0]


def make_cache(rng, pages, page, heads, dim, dtype, heads_first=False):
    cache = kv.KVCache.empty(pages, page, heads, dim, dtype, heads_first=heads_first)
    for t in (cache.k, cache.v):
        t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
    return cache


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,page,heads,dim,heads_first", [
    (1, 16, 1, 64, False), (16, 16, 20, 128, False), (37, 8, 3, 256, True), (300, 64, 5, 64, True),
    (1000, 32, 1, 128, False), (5000, 16, 8, 128, False)])
def test_write(rows, page, heads, dim, heads_first, dtype):
    rng = np.random.default_rng(rows + heads)
    pages = rows // page + 3
    cache = make_cache(rng, pages, page, heads, dim, dtype, heads_first)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    qkv = torch.from_numpy(rng.standard_normal((rows, (2 + 2) * heads * dim)).astype(np.float32)) \
        .to(dtype).cuda()
    k = qkv[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
    v = qkv[:, 2 * heads * dim:3 * heads * dim].unflatten(1, (heads, dim))
    slots = rng.permutation(pages * page)[:rows].astype(np.int64)
    slots[rng.random(rows) < 0.1] = -1
    if rows > 5:
        slots[3], slots[4] = pages * page, 1 << 40           # out of range: skipped
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, s % page], want_v[s // page, s % page] = k[t], v[t]
    kv.kv_write(cache, k, v, torch.from_numpy(slots).cuda())
    assert torch.equal(cache.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(cache.v.view(torch.int16), want_v.view(torch.int16))


def test_write_of_no_rows():
    cache = kv.KVCache.empty(2, 16, 2, 64)
    kv.kv_write(cache, cache.k[0][:0], cache.v[0][:0], ints([], torch.int64))


@pytest.mark.parametrize("requests,new,page,heads,dim,layers,heads_first", [
    (1, 1, 16, 1, 64, 1, False), (2, 8, 16, 20, 128, 3, False), (5, 64, 8, 2, 256, 2, True),
    (3, 256, 32, 1, 64, 1, False), (2, 5, 16, 1, 64, 70, False)])
def test_commit(requests, new, page, heads, dim, layers, heads_first):
    rng = np.random.default_rng(new)
    ctx = rng.integers(0, 40, requests).tolist()
    width = -(-(max(ctx) + new) // page)
    order = rng.permutation(requests * width + 2)
    table = order[:requests * width].reshape(requests, width)
    caches = [make_cache(rng, len(order), page, heads, dim, torch.bfloat16, heads_first)
              for _ in range(layers)]
    paths = [np.sort(rng.permutation(new)[:rng.integers(0, new + 1)]).tolist() for _ in range(requests)]
    if requests > 1:
        paths[1] = list(range(new))                           # every draft accepted: nothing moves
    want = [(c.k.clone(), c.v.clone()) for c in caches]
    for b, path in enumerate(paths):
        for j, p in enumerate(path):
            (s0, s1), (d0, d1) = divmod(ctx[b] + p, page), divmod(ctx[b] + j, page)
            for k, v in want:
                k[table[b, d0], d1], v[table[b, d0], d1] = k[table[b, s0], s1].clone(), v[table[b, s0], s1].clone()
    path = np.full((requests, new), -1)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    got = kv.kv_commit(caches, ints(table.tolist()), ints(ctx), ints(path.tolist()),
                       ints([len(p) for p in paths]))
    assert got.tolist() == [c + len(p) for c, p in zip(ctx, paths)]
    for c, (k, v) in zip(caches, want):
        assert torch.equal(c.k.view(torch.int16), k.view(torch.int16))
        assert torch.equal(c.v.view(torch.int16), v.view(torch.int16))


def test_commit_cuts_a_path_that_is_none():
    rng = np.random.default_rng(1)
    cache = make_cache(rng, 8, 16, 2, 64, torch.float16)
    k = cache.k.clone()
    table = ints([[0, 1], [2, 3], [4, -1], [6, 99], [7, 5]])
    ctx = ints([10, 10, 10, 10, -5])
    path = ints([[0, 2, 2, 5], [-1, 0, 1, 2], [1, 3, 9, 11], [2, 5, 6, 7], [1, 2, 3, 4]])
    got = kv.kv_commit(cache, table, ctx, path, ints([4, 4, 9, 4, 4]))
    # request 2: 10 + 9 has no page; 3: 10 + 6 neither; 4: a negative length keeps nothing
    assert got.tolist() == [12, 10, 12, 12, -5]
    k[0, 11] = k[0, 12]
    k[4, 10], k[4, 11] = k[4, 11].clone(), k[4, 13].clone()
    k[6, 10], k[6, 11] = k[6, 12].clone(), k[6, 15].clone()
    assert torch.equal(cache.k, k)


def test_a_step_in_a_graph_with_other_lengths():
    """plan and write captured once, replayed with other lengths."""
    rng = np.random.default_rng(8)
    cache = make_cache(rng, 12, 16, 2, 64, torch.bfloat16)
    ctx, new, table = ints([0, 0]), ints([1, 1]), ints([[0, 1, 2, 3], [4, 5, 6, 7]])
    free, plan = ints([8, 9, 10, 11]), kv.KVPlan.empty(2, 8)
    k = torch.randn(8, 2, 64, device="cuda").to(torch.bfloat16)
    kv.kv_plan(ctx, new, table, free, 16, 8, plan=plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kv_plan(ctx, new, table, free, 16, 8, plan=plan)
        kv.kv_write(cache, k, k, plan.slots)
    table.copy_(ints([[0, 1, -1, -1], [4, -1, -1, -1]]))
    ctx.copy_(ints([30, 16]))
    new.copy_(ints([3, 5]))
    graph.replay()
    assert table.tolist() == [[0, 1, 8, -1], [4, 9, -1, -1]]
    want = [1 * 16 + 14, 1 * 16 + 15, 8 * 16, 9 * 16, 9 * 16 + 1, 9 * 16 + 2, 9 * 16 + 3, 9 * 16 + 4]
    assert plan.slots.tolist() == want
    assert torch.equal(cache.k.flatten(0, 1)[want], k)
