"""Many rows over the 8-bit cache where values' units are unlike: rows of zeros, high scores on small values,
probabilities far below the largest.  The tile kernel against the statement in 64 bits."""

import types

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import kv
from tests import kv_reference as R
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
I8, E4 = torch.int8, torch.float8_e4m3fn
BF, HF = torch.bfloat16, torch.float16
LARGEST = {I8: 127.0, E4: 448.0}
SCALE, Q0 = 0.25, 32.0       # a key whose first element is x has 8 x more than its score otherwise
GROUP, NEW = 2, 30           # 60 rows a key head: the tile kernel's for every head size


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def given(rng, ctx, heads, dim, dtype, kind, new=NEW, spread=0.2, group=GROUP, other=0.5):
    """Tokens [ctx + new] of one request: codes (as numbers), units, queries; scores apart from the first element
    are `other` times as wide as usual."""
    n = ctx + new
    g = types.SimpleNamespace(ctx=ctx, new=new, heads=heads, dim=dim, dtype=dtype, kind=kind)
    for name in ("k", "v"):
        x = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32)).mul_(LARGEST[kind] / 7)
        x.clamp_(-LARGEST[kind], LARGEST[kind])
        if name == "k":
            x[..., 0] = 0
        setattr(g, name, x.round() if kind == I8 else x.to(E4).float())
        unit = np.exp(spread * rng.standard_normal((n, heads))) * 7 / LARGEST[kind]
        setattr(g, name + "u", torch.from_numpy(unit.astype(np.float32)))
    q = other * rng.standard_normal((new, heads * group, dim))
    q[..., 0] = Q0
    g.q = torch.from_numpy(q.astype(np.float32)).to(dtype)
    return g


def raise_score(g, at, by, head=slice(None)):
    """Key `at` scores `by` more than without its first element (nats)."""
    x = by / (SCALE * Q0) / g.ku[at, head]
    assert float(x.abs().max()) <= LARGEST[g.kind]
    g.k[at, head, 0] = x.round() if g.kind == I8 else x.to(E4).float()


def bounds(g, k, ref, weight, lse, scale):
    """Scores and sums as for the 16-bit cache (kv_reference.attention_bounds), with 8 roundings more for units and
    powers of two.  Probability times unit is rounded to fp16: 2^-11 relatively, and by 2^-25 where it has no exponent
    left, the row's largest being 2^7 at least, so by 2^-32 of the largest unit, times a code.  bf16 rows: value times
    unit is rounded to fp16 too, its unit first in two parts of which the second is off by 2^-25 of a 2^-8 or more:
    (1 + 2^-11)(1 + 2^-11 + 2^-17 + 2^-22) - 1 < 2^-10 + 2^-16, and twice by 2^-25 of the largest unit where values
    have no exponent left."""
    keys, eps, unit = g.ctx + g.new, 2.0 ** -24, R.UNIT[g.dtype]
    q = g.q.double().numpy()
    most = scale * np.sqrt((q ** 2).sum(-1)).max() * np.sqrt((k ** 2).sum(-1)).max()
    rel = (g.dim + 10) * eps * most + 2.0 ** -21 + (keys + 8) * eps
    folds, vu = g.dtype is BF, float(g.vu.max())
    out = weight * ((2.0 ** -10 + 2.0 ** -16 if folds else 2.0 ** -11) + 2 * rel) * (1 + 2.0 ** -11)
    out = out + unit * np.abs(ref) + (keys * 2.0 ** -32 * LARGEST[g.kind] + folds * 2.0 ** -24) * vu
    out = out + (2.0 ** -25 if g.dtype is HF else 0.0)
    return out, rel + 4 * eps * np.abs(np.where(np.isfinite(lse), lse, 0)) + 2.0 ** -19


def run(g, page=16, copies=1, lost=(), scale=SCALE, mask=None):
    """(out, lse) of `copies` requests that share the tokens' pages; pages `lost` of the table are none."""
    n = g.ctx + g.new
    need = -(-n // page)
    order = np.random.default_rng(0).permutation(need + 3)[:need]
    cache = kv.KVCache8.empty(need + 3, page, g.heads, g.dim, g.kind)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.view(torch.uint8).fill_(0xFF)
    pos = np.arange(n)
    pg, r = (torch.from_numpy(x).cuda() for x in (order[pos // page], pos % page))
    for codes, units, x, u in ((cache.k, cache.k_scale, g.k, g.ku), (cache.v, cache.v_scale, g.v, g.vu)):
        codes.view(I8)[pg, r] = x.to(g.kind).view(I8).cuda()
        units[pg, :, r] = u.cuda()
    table = order.copy()
    for i, p in enumerate(lost):
        table[p] = -1 if i % 2 == 0 else 1 << 20
    out, lse = kv.tree_attention(g.q.cuda().repeat(copies, 1, 1), cache, ints(np.tile(table, (copies, 1))),
                                 ints([g.ctx] * copies), ints([g.new * i for i in range(copies + 1)]), g.new,
                                 mask=mask, scale=scale, return_lse=True)
    B.tern_check()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def compare(g, copies=1, scale=SCALE, **kw):
    k, v = ((x * u[..., None]).double().numpy()[None] for x, u in ((g.k, g.ku), (g.v, g.vu)))
    ref, rl, weight = R.attention(g.q.double().numpy(), k, v, [[0]], g.ctx + g.new, [g.ctx], [g.new],
                                  lambda b, i, j: j <= i, scale)
    ob, lb = bounds(g, k, ref, weight, rl, scale)
    out, lse = run(g, copies=copies, scale=scale, **kw)
    for i in range(copies):
        o, l = out[i * g.new:(i + 1) * g.new], lse[i * g.new:(i + 1) * g.new]
        assert (np.abs(o - ref) <= ob).all(), float(np.nan_to_num(np.abs(o - ref) / ob, nan=np.inf).max())
        assert (np.abs(l - rl) <= lb).all(), float(np.nan_to_num(np.abs(l - rl) / lb, nan=np.inf).max())


KINDS = pytest.mark.parametrize("dtype,kind,dim", [(BF, I8, 64), (BF, I8, 128), (BF, E4, 128), (BF, E4, 256),
                                                   (HF, I8, 128), (HF, E4, 256)])


# ---------------------------------------------------------------- rows of zeros

@KINDS
def test_zero_filled_cache(dtype, kind, dim):
    """Nothing but zeros, as in a first step over a cleared cache."""
    g = given(np.random.default_rng(1), 1000, 2, dim, dtype, kind)
    for x in (g.k, g.v, g.ku, g.vu):
        x.zero_()
    out, lse = run(g)
    assert (out == 0).all()
    want = np.log(1001 + np.arange(NEW))[:, None]
    assert (np.abs(lse - want) <= 2.0 ** -18).all()


@KINDS
@pytest.mark.parametrize("first,last", [(0, 128), (256, 512), (872, 1000), (0, 1000)])
def test_tiles_of_zero_values(dtype, kind, dim, first, last):
    g = given(np.random.default_rng(first + dim), 1000, 2, dim, dtype, kind)
    g.v[first:last, 1], g.vu[first:last, 1] = 0, 0
    compare(g)


@KINDS
@pytest.mark.parametrize("at", [3, 700])
@pytest.mark.parametrize("by", [0.0, 9.7, 25.0])
def test_one_zero_valued_key(dtype, kind, dim, at, by):
    """One among others, scored as they are and far above them."""
    g = given(np.random.default_rng(at + dim), 1000, 2, dim, dtype, kind)
    g.v[at, 0], g.vu[at, 0] = 0, 0
    raise_score(g, at, by)
    compare(g)


@KINDS
def test_lost_pages(dtype, kind, dim):
    """Pages out of range count as zeros: some, and all of several tiles."""
    g = given(np.random.default_rng(dim), 1000, 2, dim, dtype, kind)
    lost = [0, 5] + list(range(16, 33)) + [50]
    for p in lost:
        for x in (g.k, g.v):
            x[p * 16:p * 16 + 16] = 0
    compare(g, lost=lost)


# ---------------------------------------------------------------- high scores on small values

@KINDS
@pytest.mark.parametrize("at", [3, 300, 700])
@pytest.mark.parametrize("by,smaller", [(7.0, 5), (9.4, 6), (9.4, 8), (12.0, 7), (12.0, 10), (16.0, 9), (16.0, 12)])
def test_high_score_on_a_small_value(dtype, kind, dim, at, by, smaller):
    """A key as the first tokens of a text often are: by `by` above the others (nats), its value's unit 2^-smaller of
    theirs; in an item's first tile and in later ones.  Items enough that most have one CTA."""
    g = given(np.random.default_rng(at + dim + smaller), 1000, 2, dim, dtype, kind)
    raise_score(g, at, by)
    g.vu[at] *= 2.0 ** -smaller
    compare(g, copies=48)


@KINDS
@pytest.mark.parametrize("most", [7, 9, 11, 30])
def test_scores_and_units_against_each_other(dtype, kind, dim, most):
    """Every key's value unit is down to 2^-most of the largest, and its score the higher for it, by as much or more."""
    rng = np.random.default_rng(most + dim)
    g = given(rng, 1000, 2, dim, dtype, kind, spread=0.0, other=0.1)
    down = rng.uniform(0, most, g.vu.shape)
    g.vu *= torch.from_numpy(2.0 ** -down).float()
    x = torch.from_numpy(down * np.log(2) * 1.5).float() / (SCALE * Q0) / g.ku
    g.k[..., 0] = x.round() if kind == I8 else x.to(E4).float()
    compare(g, copies=24)


@KINDS
@pytest.mark.parametrize("spread", [0.6, 0.9, 1.2, 2.0])
def test_units_apart(dtype, kind, dim, spread):
    """Tiles on both sides of where units are folded into the values, one after another."""
    compare(given(np.random.default_rng(dim), 2000, 2, dim, dtype, kind, spread=spread, other=0.2), copies=8)


# ---------------------------------------------------------------- probabilities far below the largest

@KINDS
@pytest.mark.parametrize("below", [27, 29, 31])
def test_many_keys_far_below_one(dtype, kind, dim, below):
    """One key with a value of zero in some columns, and in an item's other tiles thousands whose probability is
    2^-below of its: these columns are all theirs, and 2^-32 of the largest is what a probability may lose."""
    g = given(np.random.default_rng(below), 4000, 1, dim, dtype, kind, new=60, spread=0.0, group=1, other=0.0)
    g.k[:], g.v[:, :, :8] = 0, 0.8 * LARGEST[kind] // 16 * 16
    raise_score(g, 5, below * np.log(2))
    g.v[5, :, :8] = 0
    compare(g, copies=200)


# ---------------------------------------------------------------- sums of probabilities

@KINDS
@pytest.mark.parametrize("last", [0, 200])
def test_sums_over_many_zero_valued_keys(dtype, kind, dim, last):
    """A head whose values are zeros (but for the last cached tokens), its first tile's scores below the others': the
    reference follows scores less the log2 of a least unit, and thousands of probabilities far above it are added up."""
    g = given(np.random.default_rng(dim), 20000, 1, dim, dtype, kind, new=60, spread=0.0, group=1, other=0.0)
    g.k[:] = 0
    raise_score(g, slice(128, None), 7.5 * np.log(2))
    zero = slice(0, g.ctx - last)
    g.v[zero], g.vu[zero] = 0, 0
    if last == 0:
        g.v[:], g.vu[:] = 0, 0
    compare(g, copies=160)


# ---------------------------------------------------------------- what the kernel of few rows is tested with

@KINDS
@pytest.mark.parametrize("spread", [4.0, 8.0])
def test_units_far_apart(dtype, kind, dim, spread):
    """Units of keys and values over many orders of magnitude."""
    g = given(np.random.default_rng(dim), 900, 2, dim, dtype, kind, spread=spread, other=0.5 * np.exp(-2.5 * spread))
    g.q[..., 0] = 0
    g.vu /= float(g.vu.max())
    compare(g, copies=4)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind,dim", [(I8, 64), (E4, 128), (I8, 256)])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -9, 2.0 ** 8, 2.0 ** 14])
def test_queries_of_any_size(dtype, kind, dim, size):
    """Queries and the scale in inverse proportion: the same scores."""
    if dtype is HF and not 2.0 ** -10 < size < 2.0 ** 9:
        size = 2.0 ** (8 if size > 1 else -10)
    g = given(np.random.default_rng(3), 500, 2, dim, dtype, kind)
    g.q[..., 0] = 0
    want, wl = run(g)
    g.q = (g.q.double() * size).to(dtype)
    got, gl = run(g, scale=SCALE / size)
    if dtype is BF:              # a power of two, which the kernel takes out
        assert np.array_equal(got, want) and np.array_equal(gl, wl)
    else:
        compare(g, scale=SCALE / size)


@KINDS
@pytest.mark.parametrize("new", [3, 30])
def test_drafts_that_a_row_does_not_see_may_be_anything(dtype, kind, dim, new):
    """A draft's units NaN: its siblings' rows are the same as without, the rows that see it NaN; in both kernels."""
    g = given(np.random.default_rng(dim), 37, 2, dim, dtype, kind, new=new)
    parents = [-1, 0, 0] + [2 if i % 3 == 0 else 1 for i in range(3, new)]
    mask = kv.ancestor_masks(parents)
    want, wl = run(g, mask=mask)
    sees = [2] + [i for i in range(3, new) if i % 3 == 0]
    keep = [i for i in range(new) if i not in sees]
    g.ku[39], g.vu[39] = float("nan"), float("nan")
    got, gl = run(g, mask=mask)
    assert np.array_equal(got[keep], want[keep]) and np.array_equal(gl[keep], wl[keep])
    assert np.isnan(got[sees]).all() and np.isnan(gl[sees]).all()


@KINDS
@pytest.mark.parametrize("at", [0, 200, 999])
@pytest.mark.parametrize("unit", ["ku", "vu"])
def test_cached_token_that_is_nan(dtype, kind, dim, at, unit):
    """One head's unit of a cached token: all of that head's rows are NaN, the other head's as without."""
    g = given(np.random.default_rng(at), 1000, 2, dim, dtype, kind)
    want, wl = run(g)
    getattr(g, unit)[at, 1] = float("nan")
    got, gl = run(g)
    assert np.array_equal(got[:, :GROUP], want[:, :GROUP]) and np.array_equal(gl[:, :GROUP], wl[:, :GROUP])
    assert np.isnan(got[:, GROUP:]).all()
    assert np.isnan(gl[:, GROUP:]).all() == (unit == "ku")
