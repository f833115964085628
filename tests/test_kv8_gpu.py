"""The 8-bit cache's write, read and commit, and rows that are normalised and rotated as they are
written, against plain statements of them."""

import math

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import kv
from tests import kv8_reference as R
from tests.gpu_helpers import ensure_lib, poison
from tests.kv_reference import UNIT

pytestmark = pytest.mark.gpu
KINDS = [torch.int8, torch.float8_e4m3fn]
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8)


def make_cache8(pages, page, heads, dim, kind, heads_first=False):
    c = kv.KVCache8.empty(pages, page, heads, dim, kind, heads_first=heads_first)
    gen = torch.Generator(device="cuda").manual_seed(pages)
    for t in (c.k, c.v):
        t.view(torch.int8).copy_(torch.randint(-127, 126, t.shape, generator=gen, device="cuda", dtype=torch.int8))
    for t in (c.k_scale, c.v_scale):
        t.uniform_(0.5, 1.5, generator=gen)
    return c


def state(c):
    return [t.view(torch.int8).clone() if t.dtype != torch.float32 else t.clone()
            for t in (c.k, c.v, c.k_scale, c.v_scale)]


def put(want, slots, page, k, v, kind):
    """Rows written into copies of the cache's tensors; slots outside it are skipped."""
    pages = want[0].shape[0]
    for i, slot in enumerate(slots):
        if 0 <= slot < pages * page:
            at, r = divmod(slot, page)
            for x, codes, units in ((k, want[0], want[2]), (v, want[1], want[3])):
                c, u = R.quantise(x[i].float(), kind)
                codes[at, r], units[at, :, r] = c.view(torch.int8).to(codes.device), u.to(units.device)


def same(a, b):
    return torch.equal(a, b) if a.dtype != torch.float32 else torch.equal(a.view(torch.int32), b.view(torch.int32)) or \
        bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,page,heads,dim,heads_first,dtype", [
    (1, 16, 1, 64, False, BF), (16, 16, 20, 128, False, HF), (37, 8, 3, 256, True, BF), (300, 64, 5, 64, True, HF),
    (1000, 32, 1, 128, False, BF), (411, 256, 7, 128, False, HF)])
def test_write_and_read(rows, page, heads, dim, heads_first, dtype, kind):
    """Codes and units in the operator's own float32 steps: equal, and nothing else changes."""
    rng = np.random.default_rng(rows + heads)
    pages = rows // page + 3
    c = make_cache8(pages, page, heads, dim, kind, heads_first)
    want = [t.cpu() for t in state(c)]
    qkv = torch.from_numpy(rng.standard_normal((rows, 4 * heads * dim)).astype(np.float32)).to(dtype).cuda()
    k, v = (qkv[:, i * heads * dim:(i + 1) * heads * dim].unflatten(1, (heads, dim)) for i in (1, 3))
    slots = rng.permutation(pages * page)[:rows]
    slots[rng.random(rows) < 0.1] = -1
    if rows > 4:
        slots[2], slots[4] = pages * page, -(1 << 62)
    kv.kv_write(c, k, v, ints(slots, torch.int64))
    put(want, slots, page, k.cpu(), v.cpu(), kind)
    assert all(same(a.cpu(), b) for a, b in zip(state(c), want))
    for out in (BF, HF):
        got = kv.kv_read(c, ints(slots, torch.int64), dtype=out)
        for g, codes, units in zip(got, want[:2], want[2:]):
            inside = (slots >= 0) & (slots < pages * page)
            at = np.where(inside, slots, 0)
            ref = codes[at // page, at % page].view(kind).float() * units[at // page, :, at % page][..., None]
            ref[~inside] = 0
            assert torch.equal(g.cpu(), ref.to(out))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_are_not_ordinary(kind):
    x = torch.zeros(9, 2, 64, dtype=BF)
    x[1] = 2.0 ** -110
    x[2, :, 3] = math.inf
    x[3, :, 3] = math.nan
    x[4] = 3e38
    x[5, 0, 7], x[5, 1] = -1.0, 2.0 ** -99
    x[6, :, :2] = torch.tensor([1e30, 1e-30])
    x[7] = torch.linspace(-127, 127, 64)
    x[8, 0, 0], x[8, 1, 63] = -math.inf, 2.0 ** -100
    c = make_cache8(2, 8, 2, 64, kind)
    want = [t.cpu() for t in state(c)]
    kv.kv_write(c, x.cuda(), x.flip(0).cuda(), ints(range(9), torch.int64))
    put(want, range(9), 8, x, x.flip(0), kind)
    assert all(same(a.cpu(), b) for a, b in zip(state(c), want))
    k, _ = kv.kv_read(c, ints(range(9), torch.int64))
    assert (k[0] == 0).all() and (k[1] == 0).all() and k[2].isnan().all() and k[3].isnan().all()
    assert torch.isfinite(k[4]).all() and k[8, 0].isnan().all() and (k[8, 1, 63] > 0)


def rotate_bound(x, norm, dim, ref):
    """What roundings add up to before the last: the mean's (dim + 2) 2^-24 halved by the root, rsqrt and two
    products (4 2^-24), and of the rotation cosines and sines off by 2^-22 (angle to 2^-25 of a turn's half,
    sincospif 2 ulp) and three operations, times both elements of the pair; |pair| <= sqrt 2 of the largest."""
    largest = ref.abs().amax(-1, keepdim=True) + 2.0 ** -120
    return largest * ((dim + 2) / 2 + 4 + 4 + 8 + 3) * 2.0 ** -24 * 1.5


@pytest.mark.parametrize("kind", [None] + KINDS)
@pytest.mark.parametrize("rows,hq,heads,dim,rot,axes,neighbours,norm,dtype", [
    (1, 1, 1, 64, 64, 1, False, "rows", BF), (16, 40, 20, 128, 128, 1, False, "f32", BF),
    (37, 6, 3, 256, 64, 3, False, "rows", HF), (130, 5, 5, 64, 16, 2, True, None, HF),
    (3, 33, 11, 128, 80, 3, True, "rows", BF), (1200, 4, 2, 128, 0, 1, False, "rows", BF),
    (700, 8, 1, 256, 256, 1, False, None, BF), (5, 3, 1, 64, 48, 1, False, "q", HF)])
def test_rotate_write(rows, hq, heads, dim, rot, axes, neighbours, norm, dtype, kind):
    rng = np.random.default_rng(rows + dim)
    gen = torch.Generator().manual_seed(rows)
    page, pages = 16, rows // 16 + 2
    c = kv.KVCache.empty(pages, page, heads, dim, dtype) if kind is None else make_cache8(pages, page, heads, dim, kind)
    if kind is None:
        for t in (c.k, c.v):
            t.copy_(torch.randn(t.shape, generator=gen))
    before = [t.clone() for t in (c.k, c.v)]
    qkv = torch.randn(rows, (hq + 2 * heads) * dim, generator=gen).mul_(3).to(dtype)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([hq * dim, heads * dim, heads * dim], 1))
    weights = [None, None]
    if norm is not None:
        weights = [(1 + 0.2 * torch.randn(dim, generator=gen)).to(torch.float32 if norm == "f32" else dtype)
                   for _ in range(2)]
        if norm == "q":
            weights[1] = None
    freq = [1e4 ** (-2 * j / rot) if j else 1.0 for j in range(rot // 2)]
    axis = [j % axes for j in range(rot // 2)] if axes > 1 else None
    positions = torch.from_numpy(rng.integers(0, 200000, (axes, rows)))
    positions[:, 0] = 0
    if rows > 2:
        positions[0, 1], positions[0, 2] = 2 ** 31 - 1, -77
    rotary = kv.Rotary(freq, axis=axis, neighbours=neighbours) if rot else None
    slots = rng.permutation(pages * page)[:rows]
    if rows > 1:
        slots[1] = -1
    at = positions.int().cuda()
    dev = [None if w is None else w.cuda() for w in weights]
    cuda = qkv.cuda()
    qd, kd, vd = (t.unflatten(1, (-1, dim)) for t in cuda.split([hq * dim, heads * dim, heads * dim], 1))
    out = kv.rotate_write(c, qd, kd, vd, ints(slots, torch.int64), rotary, (at if axes > 1 else at[0]) if rot else None,
                          dev[0], dev[1])
    unit = UNIT[dtype]
    # positions of 2^31 turn an angle's last bits of 64: the reference keeps 53 (2^31 2^-53 2^2)
    far = 2.0 ** -20
    ref = R.rotate(q, weights[0], 1e-6, freq, axis, positions, neighbours)
    bound = rotate_bound(q, weights[0], dim, ref) + unit * ref.abs()
    if rows > 2:
        bound[1] += ref[1].abs().amax() * far
    assert ((out.cpu().double() - ref).abs() <= bound + 2.0 ** -24).all()
    inside = slots >= 0
    at, r = slots[inside] // page, slots[inside] % page
    ref = R.rotate(k, weights[1], 1e-6, freq, axis, positions, neighbours)
    bound = rotate_bound(k, weights[1], dim, ref)
    if rows > 2:
        bound[1] += ref[1].abs().amax() * far
    if kind is None:
        assert ((c.k.cpu()[at, r].double() - ref[inside]).abs() <= (bound + unit * ref.abs() + 2.0 ** -24)[inside]).all()
        assert torch.equal(c.v.cpu()[at, r], v[inside])
        free = np.setdiff1d(np.arange(pages * page), slots)
        for t, b in zip((c.k, c.v), before):
            assert torch.equal(t.cpu()[free // page, free % page], b.cpu()[free // page, free % page])
        return
    # a code is off by half a step: of int8 1/2, of e4m3 2^-4 of itself and 2^-10 at least; and the unit and
    # the value as the rotation rounds them
    codes = c.k.view(torch.int8).cpu()[at, r].view(kind).double()
    units = c.k_scale.cpu()[at, :, r].double()[..., None]
    most = ref[inside].abs().amax(-1, keepdim=True)
    assert ((units * R.LARGEST[kind] - most).abs() <= bound[inside].amax(-1, keepdim=True) + most * 2.0 ** -22).all()
    step = 0.5 if kind == torch.int8 else torch.maximum(codes.abs() * 2.0 ** -3.5, torch.tensor(2.0 ** -10))
    assert ((codes * units - ref[inside]).abs() <= step * units * (1 + 2.0 ** -20) + 2 * bound[inside]).all()
    want = [t.cpu() for t in state(c)]
    put(want, slots, page, torch.zeros_like(k), v, kind)
    assert same(c.v.view(torch.int8).cpu(), want[1]) and same(c.v_scale.cpu(), want[3])


def test_rotate_write_in_place_and_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(33, 6, 128, generator=gen, device="cuda").to(BF)
    k = torch.randn(33, 2, 128, generator=gen, device="cuda").to(BF)
    rotary, at = kv.Rotary.geometric(128), torch.arange(33, dtype=torch.int32, device="cuda")
    caches = [kv.KVCache.empty(4, 16, 2, 128) for _ in range(2)]
    slots = torch.arange(33, device="cuda")
    a = kv.rotate_write(caches[0], q, k, k, slots, rotary, at)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = kv.rotate_write(caches[1], q, k, k, slots, rotary, at, stream=side)
    kv.rotate_write(caches[1], q, k, k, slots, rotary, at, out=q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, q)
    assert torch.equal(caches[0].k.flatten(0, 1)[:33], caches[1].k.flatten(0, 1)[:33])


def test_no_rows():
    c = make_cache8(2, 16, 1, 64, torch.int8)
    before = state(c)
    none = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    kv.kv_write(c, none, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    k, v = kv.kv_read(c, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert k.shape == v.shape == (0, 1, 64) and all(same(a, b) for a, b in zip(state(c), before))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layers,heads,dim,page", [(1, 1, 64, 8), (3, 5, 128, 16), (35, 20, 256, 32)])
def test_commit(layers, heads, dim, page, kind):
    rng = np.random.default_rng(layers)
    ctx, new = [3, 0, 3 * page - 1, 17], [9, 6, 12, 1]
    width = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 1
    pages = 4 * width + 2
    order = rng.permutation(pages)
    table = [[int(order[b * width + i]) for i in range(width)] for b in range(4)]
    caches = [make_cache8(pages, page, heads, dim, kind) for _ in range(layers)]
    want = [state(c) for c in caches]
    path = [[0, 2, 3, 8], [1, 4, 4, 5], [0, 1, 2, 3], [0, 0, 0, 0]]
    length, kept = [4, 4, 4, 1], [4, 2, 4, 1]
    got = kv.kv_commit(caches, ints(table), ints(ctx), ints(path), ints(length))
    assert got.tolist() == [c + n for c, n in zip(ctx, kept)]
    for w in want:
        for b, c in enumerate(ctx):
            for j in range(kept[b]):
                f, t = c + path[b][j], c + j
                pf, pt = table[b][f // page], table[b][t // page]
                for x in w[:2]:
                    x[pt, t % page] = x[pf, f % page].clone()
                for x in w[2:]:
                    x[pt, :, t % page] = x[pf, :, f % page].clone()
    for c, w in zip(caches, want):
        assert all(same(a, b) for a, b in zip(state(c), w))


def test_commit_of_both_kinds_is_refused():
    with pytest.raises(ValueError, match="all of 16 bits or all of 8"):
        kv.kv_commit([kv.KVCache.empty(2, 16, 1, 64), kv.KVCache8.empty(2, 16, 1, 64)], ints([[0]]), ints([0]),
                     ints([[0]]), ints([1]))


def test_refusals():
    c = kv.KVCache8.empty(2, 16, 2, 64)
    k = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    slots = ints([0, 1, 2], torch.int64)
    at = ints([0, 1, 2])
    three = kv.Rotary([1.0] * 8, axis=[0, 1, 2, 0, 1, 2, 0, 1])
    for what, call in [
            ("k: expected bf16", lambda: kv.kv_write(c, k.float(), k.float(), slots)),
            ("k: expected", lambda: kv.kv_write(c, k[:, :1], k, slots)),
            ("v: expected", lambda: kv.kv_write(c, k, k.half(), slots)),
            ("slots", lambda: kv.kv_write(c, k, k, slots[:2])),
            ("cache's type", lambda: kv.rotate_write(kv.KVCache.empty(2, 16, 2, 64, HF), None, k, k, slots)),
            ("positions: expected with", lambda: kv.rotate_write(c, k, k, k, slots, three)),
            ("several axes", lambda: kv.rotate_write(c, k, k, k, slots, three, at)),
            ("axes, rows", lambda: kv.rotate_write(c, k, k, k, slots, three, at.expand(3, 3)[:, :2])),
            ("one each row", lambda: kv.rotate_write(c, k, k, k, slots, kv.Rotary([1.0] * 8), at[:2])),
            ("than a head has", lambda: kv.rotate_write(c, k, k, k, slots, kv.Rotary([1.0] * 40), at)),
            ("q_norm", lambda: kv.rotate_write(c, k, k, k, slots, q_norm=torch.ones(63, dtype=BF, device="cuda"))),
            ("q_norm", lambda: kv.rotate_write(c, k, k, k, slots, q_norm=torch.ones(64, dtype=HF, device="cuda"))),
            ("k_norm", lambda: kv.rotate_write(c, k, k, k, slots, q_norm=torch.ones(64, device="cuda"),
                                               k_norm=torch.ones(64, dtype=BF, device="cuda"))),
            ("out: expected", lambda: kv.rotate_write(c, k, k, k, slots, out=k[:2])),
            ("8-bit", lambda: kv.kv_read(kv.KVCache.empty(2, 16, 2, 64), slots)),
            ("dtype", lambda: kv.kv_read(c, slots, dtype=torch.float32)),
            ("slot each row", lambda: kv.kv_read(c, slots, k=torch.zeros(4, 2, 64, dtype=BF, device="cuda"))),
            ("k: expected", lambda: kv.KVCache8(k, k, k, k)),
            ("k_scale", lambda: kv.KVCache8(c.k, c.v, c.k_scale[:1], c.v_scale))]:
        with pytest.raises(ValueError, match=what):
            call()
