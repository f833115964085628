"""Tree attention over the 8-bit cache against its statement in 64 bits."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu
I8, E4 = torch.int8, torch.float8_e4m3fn
BF, HF = torch.bfloat16, torch.float16
LARGEST = {I8: 127.0, E4: 448.0}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def bounds(q, k, dim, keys, scale, dtype, ref, weight, lse, unit_most, largest):
    """As for the 16-bit cache, with the roundings that differ: probabilities times units to fp16 (2^-11
    relatively, 2^-32 of the row's largest where they have no exponent left, times codes up to `largest`), the
    score's units and powers of two (8 in all), the queries as they are.  For bf16 rows the many-row kernel may
    also round value * unit / 2^E to fp16, unit / 2^E in [2^-10, 2): relatively 2^-11, so that both roundings give
    (1 + 2^-11)^2 - 1 < 2^-10 (1 + 2^-11), and where it has no exponent left by 2^-25 2^E <= 2^-25 of the largest
    unit for a row whose probabilities sum to 1."""
    unit, eps = R.UNIT[dtype], 2.0 ** -24
    most = abs(scale) * np.sqrt((q ** 2).sum(-1)).max() * np.sqrt((k ** 2).sum(-1)).max()
    rel = (dim + 10) * eps * most + 2.0 ** -21 + (keys + 8) * eps
    folds = dtype is BF
    out = weight * (2.0 ** (-10 if folds else -11) + 2 * rel) * (1 + 2.0 ** -11) + unit * np.abs(ref) + 2.0 ** -24
    out = out + (keys * 2.0 ** -32 * largest + folds * 2.0 ** -25) * unit_most
    return out, rel + 4 * eps * np.abs(np.where(np.isfinite(lse), lse, 0)) + 2.0 ** -19


def make(rng, ctx, new, page, heads, group, dim, dtype, kind, heads_first=False, spread=0.3, spare=1, fill=0xFF):
    """A cache whose bytes past the requests' last tokens are what `fill` gives (of e4m3 and of the units NaN)."""
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    width, pages = max(need + [1]) + spare, sum(need) + 3
    order = rng.permutation(pages)
    table, at = np.full((len(ctx), width), -1), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = kv.KVCache8.empty(pages, page, heads, dim, kind, heads_first=heads_first)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.view(torch.uint8).fill_(fill) if t.is_contiguous() else t.view(torch.int8).fill_(-1 if fill == 0xFF else 0)
    k, v = (torch.zeros(pages, page, heads, dim) for _ in range(2))
    pos = [(table[b, p // page], p % page) for b, (c, n) in enumerate(zip(ctx, new)) for p in range(c + n)]
    if pos:
        pg, r = (torch.tensor(x, device="cuda") for x in zip(*pos))
        for x, codes, units in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
            val = rng.standard_normal((len(pos), heads, dim)).astype(np.float32)
            if x is k:
                val[..., :3] += 3
            val = torch.from_numpy(val).mul_(LARGEST[kind] / 7).clamp_(-LARGEST[kind], LARGEST[kind])
            code = val.round().to(I8) if kind == I8 else val.to(E4)
            unit = torch.from_numpy(np.exp(spread * rng.standard_normal((len(pos), heads))).astype(np.float32)) * \
                (7 / LARGEST[kind])
            codes.view(I8)[pg, r] = code.view(I8).cuda()
            units[pg, :, r] = unit.cuda()
            x[pg.cpu(), r.cpu()] = code.float() * unit[..., None]
            assert torch.isfinite(x).all()
    t = sum(new)
    q = torch.from_numpy(rng.standard_normal((t, heads * group, dim)).astype(np.float32)).to(dtype)
    starts = np.concatenate([[0], np.cumsum(new)])
    return cache, k.double().numpy(), v.double().numpy(), table, q, starts


def check(rng, ctx, new, page, heads, group, dim, dtype, kind, masks=None, scale=None, ws=None, **kw):
    cache, k, v, table, q, starts = make(rng, ctx, new, page, heads, group, dim, dtype, kind, **kw)
    t, words = sum(new), max(1, -(-max(new) // 64))
    seen = masks or (lambda b, i, j: j <= i)
    mask = None
    if masks is not None:
        rows = [[sum(1 << (j % 64) for j in range(w * 64, min(n, w * 64 + 64)) if seen(b, i, j)) for w in range(words)]
                for b, n in enumerate(new) for i in range(n)]
        mask = ints(np.array(rows, dtype=np.uint64).astype(np.int64).reshape(t, words), torch.int64)
    scale = dim ** -0.5 if scale is None else scale
    # rows behind the last stay as they were
    wide = torch.cat([q, q[:2]]) if t > 1 else q
    out = poison(torch.empty(wide.shape, dtype=dtype, device="cuda"))
    lse = poison(torch.empty(wide.shape[:2], device="cuda"))
    if mask is not None and len(wide) > t:
        mask = torch.cat([mask, mask[:2]])
    kv.tree_attention(wide.cuda(), cache, ints(table), ints(ctx), ints(starts), max(new), mask=mask, scale=scale,
                      out=out, return_lse=True, lse=lse, ws=ws)
    B.tern_check()
    ref, rl, weight = R.attention(q.double().numpy(), k, v, table, page, ctx, new, seen, scale)
    keys = max(c + n for c, n in zip(ctx, new))
    units = cache.v_scale[torch.isfinite(cache.v_scale)]
    ob, lb = bounds(q.double().numpy(), k, dim, keys, scale, dtype, ref, weight, rl,
                    float(units.max()) if units.numel() else 0.0, LARGEST[kind])
    got, gl = out[:t].double().cpu().numpy(), lse[:t].double().cpu().numpy()
    assert np.array_equal(np.isinf(gl), np.isinf(rl))
    assert (np.abs(got - ref) <= ob).all(), float((np.abs(got - ref) / ob).max())
    fin = np.isfinite(rl)
    assert (np.abs(gl[fin] - rl[fin]) <= lb[fin]).all()
    assert (got[~fin] == 0).all()
    assert (out[t:].view(torch.uint8) == 0xFF).all() and (lse[t:].view(torch.uint8) == 0xFF).all()
    return out[:t], lse[:t]


CASES = [  # ctx, new, page, heads, group, dim
    ([0], [1], 16, 1, 1, 64), ([1], [1], 8, 1, 1, 128), ([15, 16, 17, 0], [1, 1, 1, 1], 16, 2, 1, 128),
    ([63, 64, 65], [1, 2, 1], 16, 1, 8, 64), ([700, 3, 250], [1, 1, 1], 16, 3, 2, 128),
    ([127, 128], [4, 1], 256, 2, 1, 256), ([500], [4], 64, 2, 6, 256), ([333, 40], [5, 3], 8, 2, 4, 128),
    ([90, 1000, 0], [16, 3, 7], 32, 2, 5, 64), ([77], [40], 16, 1, 3, 128), ([200, 5], [29, 11], 128, 2, 8, 256),
    ([10, 0, 30], [130, 256, 1], 16, 1, 1, 64), ([50] * 40, [1] * 40, 16, 1, 4, 128), ([3000], [2], 16, 1, 130, 64)]


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chains(case, dtype, kind):
    check(np.random.default_rng(case), *CASES[case], dtype, kind)


@pytest.mark.parametrize("kind,dtype", [(I8, BF), (E4, HF)])
@pytest.mark.parametrize("ctx,new,page,heads,group,dim,heads_first", [
    ([100, 0, 31], [7, 9, 20], 16, 2, 3, 128, True), ([64], [70], 32, 1, 2, 64, False),
    ([1000, 17], [16, 5], 8, 2, 1, 256, True)])
def test_masks(ctx, new, page, heads, group, dim, heads_first, kind, dtype):
    rng = np.random.default_rng(sum(ctx))
    table = {(b, i, j): bool(rng.random() < 0.5) for b, n in enumerate(new) for i in range(n) for j in range(n)}
    for j in range(new[-1]):
        table[len(new) - 1, 2, j] = False               # a row that sees none of the new tokens
    check(rng, ctx, new, page, heads, group, dim, dtype, kind, masks=lambda b, i, j: table[b, i, j],
          heads_first=heads_first)


def test_rows_that_see_nothing():
    out, lse = check(np.random.default_rng(1), [0, 0, 40], [3, 20, 2], 16, 2, 4, 128, BF, I8,
                     masks=lambda b, i, j: b == 2 or (i + j) % 3 == 0 and i != 1)
    assert (out[1] == 0).all() and (lse[1] == -torch.inf).all()


@pytest.mark.parametrize("kind", [I8, E4])
def test_units_far_apart(kind):
    """Units over many orders of magnitude: probabilities times units keep their bits."""
    check(np.random.default_rng(5), [900, 64], [3, 1], 16, 2, 2, 128, HF, kind, spread=4.0, scale=1e-3)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 14])
def test_queries_of_any_size(size, dtype):
    rng = np.random.default_rng(6)
    cache, k, v, table, q, starts = make(rng, [80], [4], 16, 1, 4, 128, dtype, I8)
    if dtype == HF:
        size = min(max(size, 2.0 ** -10), 2.0 ** 8)
    q = (q.float() * size).to(dtype)
    out, lse = kv.tree_attention(q.cuda(), cache, ints(table), ints([80]), ints(starts), 4, scale=0.09 / size,
                                 return_lse=True)
    ref, rl, weight = R.attention(q.double().numpy(), k, v, table, 16, [80], [4], lambda b, i, j: j <= i, 0.09 / size)
    ob, lb = bounds(q.double().numpy(), k, 128, 84, 0.09 / size, dtype, ref, weight, rl,
                    float(cache.v_scale[cache.v_scale == cache.v_scale].max()), 127.0)
    assert (np.abs(out.double().cpu().numpy() - ref) <= ob).all()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= lb).all()


@pytest.mark.parametrize("kind", [I8, E4])
def test_tokens_that_a_row_does_not_see_may_be_anything(kind):
    """A draft's units NaN or infinite, its siblings' rows the same as without; a row that sees it is NaN."""
    rng = np.random.default_rng(7)
    cache, k, v, table, q, starts = make(rng, [37], [4], 16, 2, 2, 128, BF, kind)
    mask = kv.ancestor_masks([-1, 0, 0, 1])
    args = q.cuda(), cache, ints(table), ints([37]), ints(starts), 4
    want, wl = kv.tree_attention(*args, mask=mask, return_lse=True)
    pos = 37 + 2
    for unit in (cache.k_scale, cache.v_scale):
        unit[table[0, pos // 16], :, pos % 16] = float("nan")
    got, gl = kv.tree_attention(*args, mask=mask, return_lse=True)
    keep = [0, 1, 3]
    assert torch.equal(got[keep], want[keep]) and torch.equal(gl[keep], wl[keep])
    assert got[2].isnan().all() and gl[2].isnan().all()


def test_pages_out_of_range_count_as_zeros():
    rng = np.random.default_rng(8)
    for dim, page in ((128, 16), (256, 64), (64, 8)):
        cache, k, v, table, q, starts = make(rng, [200], [2], page, 1, 2, dim, BF, I8)
        lost = [1, 3] if page <= 16 else [1]
        for i in lost:
            k[table[0, i]], v[table[0, i]] = 0, 0
        bad = table.copy()
        bad[0, lost[0]] = -1
        if len(lost) > 1:
            bad[0, lost[1]] = 1 << 20
        out, lse = kv.tree_attention(q.cuda(), cache, ints(bad), ints([200]), ints(starts), 2, return_lse=True)
        B.tern_check()
        scale = dim ** -0.5
        ref, rl, weight = R.attention(q.double().numpy(), k, v, table, page, [200], [2], lambda b, i, j: j <= i, scale)
        ob, lb = bounds(q.double().numpy(), k, dim, 202, scale, BF, ref, weight, rl,
                        float(cache.v_scale[cache.v_scale == cache.v_scale].max()), 127.0)
        assert (np.abs(out.double().cpu().numpy() - ref) <= ob).all()
        assert (np.abs(lse.double().cpu().numpy() - rl) <= lb).all()


def test_long_context_of_few_heads():
    """One item over every CTA: pieces joined in groups."""
    check(np.random.default_rng(9), [20000], [3], 64, 1, 2, 64, HF, E4)
    check(np.random.default_rng(10), [9000], [1], 16, 1, 4, 256, BF, I8)


@pytest.mark.parametrize("dim,page,kind,dtype", [(128, 32, I8, BF), (64, 16, E4, HF), (256, 64, I8, HF),
                                                 (128, 256, E4, BF)])
def test_many_tiles_of_many_rows(dim, page, kind, dtype):
    """Every ring of the tile kernel goes round many times, over several items."""
    check(np.random.default_rng(dim), [3001, 640, 5], [5, 12, 3], page, 2, 6, dim, dtype, kind)
    check(np.random.default_rng(dim + 1), [9000], [70], page, 1, 1, dim, dtype, kind)


@pytest.mark.parametrize("dim,group,new", [(64, 4, 15), (64, 1, 60), (128, 4, 9), (256, 2, 10), (64, 8, 8), (64, 2, 9)])
def test_many_items_of_few_tiles(dim, group, new):
    """Items of one to four tiles one after another in a CTA: what is held of a tile is held until all have it."""
    rng = np.random.default_rng(dim + new)
    ctx = [int(c) for c in rng.integers(0, 400, 24)]
    check(rng, ctx, [int(n) for n in rng.integers(1, new + 1, 24)], 16, 8, group, dim, BF, I8)


def test_same_result_each_time_and_on_streams():
    rng = np.random.default_rng(11)
    cache, k, v, table, q, starts = make(rng, [3000, 20, 700], [3, 1, 2], 16, 2, 4, 128, BF, I8)
    args = q.cuda(), cache, ints(table), ints([3000, 20, 700]), ints(starts), 3
    ws = [B.Workspace() for _ in range(2)]
    want = kv.tree_attention(*args, ws=ws[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a = kv.tree_attention(*args, ws=ws[0])
        b = kv.tree_attention(*args, ws=ws[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_workspace_shared_with_the_16_bit_call():
    rng = np.random.default_rng(12)
    cache, k, v, table, q, starts = make(rng, [3000], [2], 16, 2, 4, 128, BF, I8)
    plain = kv.KVCache.empty(cache.pages, 16, 2, 128)
    plain.k.copy_(torch.from_numpy(k)), plain.v.copy_(torch.from_numpy(v))
    args = ints(table), ints([3000]), ints(starts), 2
    ws = B.Workspace()
    first = kv.tree_attention(q.cuda(), cache, *args, ws=ws), kv.tree_attention(q.cuda(), plain, *args, ws=ws)
    again = kv.tree_attention(q.cuda(), cache, *args, ws=ws), kv.tree_attention(q.cuda(), plain, *args, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    # 16-bit values are the codes' rounded once (2^-8), so the two differ by little
    assert float((first[0].float() - first[1].float()).norm() / first[1].float().norm()) < 0.02


def test_captured_and_replayed_with_other_lengths():
    rng = np.random.default_rng(13)
    cache, k, v, table, q, starts = make(rng, [900, 300], [2, 2], 16, 1, 4, 128, BF, E4)
    qd, td, sd, ctx = q.cuda(), ints(table), ints(starts), ints([900, 300])
    ws = B.Workspace()
    kv.tree_attention(qd, cache, td, ctx, sd, 2, ws=ws)
    out = torch.empty_like(qd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kv.tree_attention(qd, cache, td, ctx, sd, 2, out=out, ws=ws)
    for lengths in ([900, 300], [5, 299], [640, 0]):
        ctx.copy_(ints(lengths))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kv.tree_attention(qd, cache, td, ints(lengths), sd, 2))


def test_refusals():
    c = kv.KVCache8.empty(2, 16, 2, 64)
    q = torch.zeros(1, 4, 64, dtype=BF, device="cuda")
    args = ints([[0, 1]]), ints([5]), ints([0, 1]), 1
    with pytest.raises(ValueError, match="q: expected bf16"):
        kv.tree_attention(q.float(), c, *args)
    with pytest.raises(ValueError, match="multiple"):
        kv.tree_attention(q[:, :3], c, *args)
    with pytest.raises(ValueError, match="out"):
        kv.tree_attention(q, c, *args, out=torch.zeros(1, 4, 64, dtype=HF, device="cuda"))
    with pytest.raises(B.TernError):
        kv.tree_attention(q, c, *args[:3], 257)
