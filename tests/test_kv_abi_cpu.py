"""Host-side refusals of the paged-cache and tree-attention calls (no GPU needed)."""

import ctypes

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import build as BUILD
from ternary_weight_linear_block_gb300 import kv

FAKE = 1 << 20          # an aligned, never dereferenced address
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.ensure_built()
    return B.lib()


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, pages=4, page_size=16, heads=2, dim=64, page_stride=2048,
             token_stride=128, head_stride=64, dtype=0)
    d.update(kw)
    return B.KVCacheDesc(*(d[n] for n, _ in B.KVCacheDesc._fields_))


BAD_CACHES = [(dict(dtype=2), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
              (dict(k=FAKE + 8), ALIGN), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
              (dict(page_size=4), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=512), SHAPE),
              (dict(dim=96), SHAPE), (dict(heads=0), SHAPE), (dict(page_stride=2044), ALIGN),
              (dict(token_stride=0), ALIGN), (dict(head_stride=1 << 39), ALIGN)]


def st(fn, *args):
    return getattr(B.lib(), fn)(*args)


def test_plan_arguments():
    def p(ctx=FAKE, new=FAKE, b=4, page=16, table=FAKE, stride=8, width=8, free=FAKE, n_free=10,
          head=None, start=FAKE, cap=64, slots=FAKE, pos=FAKE, req=FAKE, info=FAKE, held=None,
          held_out=None):
        return st("tern_kv_plan", ctx, new, b, page, table, stride, width, held, free, n_free, head,
                  start, cap, slots, pos, req, held_out, info, None)
    for bad, want in [(dict(b=-1), INVALID), (dict(cap=-1), INVALID), (dict(n_free=-1), INVALID),
                      (dict(page=0), SHAPE), (dict(page=24), SHAPE), (dict(page=1 << 17), SHAPE),
                      (dict(b=8193), SHAPE), (dict(held=FAKE, held_out=FAKE), INVALID), (dict(cap=1 << 31), SHAPE), (dict(n_free=1 << 31), SHAPE),
                      (dict(stride=7), SHAPE), (dict(width=-1), SHAPE),
                      (dict(width=1 << 28, stride=1 << 28), SHAPE), (dict(ctx=None), INVALID),
                      (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
                      (dict(start=None), INVALID), (dict(info=None), INVALID), (dict(slots=None), INVALID),
                      (dict(slots=FAKE + 8), ALIGN), (dict(pos=FAKE + 4), ALIGN), (dict(req=FAKE + 4), ALIGN)]:
        assert p(**bad) == want, bad


def test_plan_refuses_its_own_next_head():
    # every CTA reads free_head while one writes info
    for head in (FAKE, FAKE + 8, FAKE + 12):
        assert st("tern_kv_plan", FAKE, FAKE, 4, 16, FAKE, 8, 8, None, FAKE, 10, head, FAKE, 64, FAKE, FAKE,
                  FAKE, None, FAKE, None) == INVALID, head


def test_write_arguments():
    def w(c=None, k=FAKE, v=FAKE, s=(128, 64, 128, 64), slots=FAKE, t=3):
        c = c or cache()             # kept alive while its address is in use
        return st("tern_kv_write", ctypes.addressof(c), k, v, *s, slots, t, None)
    assert st("tern_kv_write", None, FAKE, FAKE, 128, 64, 128, 64, FAKE, 3, None) == INVALID
    for bad, want in BAD_CACHES:
        assert w(cache(**bad)) == want, bad
    assert w(t=-1) == INVALID and w(t=1 << 31) == SHAPE and w(t=0) == OK
    assert w(k=None) == INVALID and w(v=None) == INVALID and w(slots=None) == INVALID
    assert w(k=FAKE + 2) == ALIGN and w(s=(100, 64, 128, 64)) == ALIGN and w(s=(128, 64, 128, -8)) == ALIGN


def test_commit_arguments():
    def c(caches=(cache(),), layers=None, b=2, table=FAKE, stride=8, width=8, ctx=FAKE, path=FAKE, pw=4,
          plen=FAKE, out=FAKE + 64):
        array = (B.KVCacheDesc * len(caches))(*caches)
        return st("tern_kv_commit", ctypes.addressof(array), len(caches) if layers is None else layers,
                  table, stride, width, ctx, path, pw, plen, out, b, None)
    for bad, want in BAD_CACHES:
        assert c((cache(), cache(**bad))) == want, bad
    assert c((cache(), cache(pages=5))) == SHAPE and c((cache(), cache(token_stride=256))) == SHAPE
    assert c(layers=0) == INVALID and c(b=-1) == INVALID and c(pw=-1) == INVALID
    assert c(b=0) == OK and c(b=65536) == SHAPE and c(pw=257) == SHAPE and c(stride=4) == SHAPE
    assert c(ctx=None) == INVALID and c(path=None) == INVALID and c(plen=None) == INVALID
    assert c(out=None) == INVALID and c(out=FAKE) == INVALID and c(table=None) == INVALID


def test_attention_arguments():
    need = B.tern_tree_attention_workspace_bytes(8, 4, 2, 64)
    assert need > B.TERN_TREE_ATTENTION_ZERO_BYTES

    def a(c=None, q=FAKE, qs=(256, 64), table=FAKE, stride=8, width=8, ctx=FAKE, start=FAKE, mask=FAKE,
          words=1, b=2, t=9, hq=4, new=8, scale=0.125, out=FAKE, lse=None, ws=FAKE, nb=need):
        c = c or cache()
        return st("tern_tree_attention", q, *qs, ctypes.addressof(c), table, stride, width, ctx,
                  start, mask, words, b, t, hq, new, scale, out, lse, ws, nb, None)
    for bad, want in BAD_CACHES:
        assert a(cache(**bad)) == want, bad
    for bad, want in [(dict(b=-1), INVALID), (dict(t=-1), INVALID), (dict(words=-1), INVALID),
                      (dict(new=-1), INVALID), (dict(scale=float("nan")), INVALID),
                      (dict(scale=float("inf")), INVALID), (dict(hq=0), SHAPE), (dict(hq=5), SHAPE),
                      (dict(b=65537), SHAPE), (dict(new=257), SHAPE), (dict(words=5), SHAPE),
                      (dict(stride=4), SHAPE), (dict(t=1 << 27), SHAPE), (dict(q=None), INVALID),
                      (dict(ctx=None), INVALID), (dict(start=None), INVALID), (dict(out=None), INVALID),
                      (dict(table=None), INVALID), (dict(words=0), INVALID), (dict(q=FAKE + 8), ALIGN),
                      (dict(out=FAKE + 8), ALIGN), (dict(qs=(250, 64)), ALIGN), (dict(ws=None), WORKSPACE),
                      (dict(nb=need - 1), WORKSPACE), (dict(ws=FAKE + 8), ALIGN), (dict(b=0), OK),
                      (dict(t=0), OK), (dict(new=0), OK)]:
        assert a(**bad) == want, bad


def test_workspace_sizes():
    ask = B.tern_tree_attention_workspace_bytes
    for bad in [(0, 4, 2, 64), (257, 4, 2, 64), (1, 4, 0, 64), (1, 3, 2, 64), (1, 1, 2, 64), (1, 4, 2, 96)]:
        assert ask(*bad) == 0, bad
    assert ask(1, 4, 4, 64) < ask(16, 4, 4, 64) < ask(64, 8, 2, 64)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_are_unsupported():
    kept = cache()
    c = ctypes.addressof(kept)
    nb = B.tern_tree_attention_workspace_bytes(8, 4, 2, 64)
    assert st("tern_kv_plan", FAKE, FAKE, 4, 16, FAKE, 8, 8, None, FAKE, 10, None, FAKE, 64, FAKE, FAKE,
              FAKE, None, FAKE, None) == UNSUPPORTED
    assert st("tern_kv_write", c, FAKE, FAKE, 128, 64, 128, 64, FAKE, 3, None) == UNSUPPORTED
    assert st("tern_kv_commit", c, 1, FAKE, 8, 8, FAKE, FAKE, 4, FAKE, FAKE + 64, 2, None) == UNSUPPORTED
    assert st("tern_tree_attention", FAKE, 256, 64, c, FAKE, 8, 8, FAKE, FAKE, None, 0, 2, 9, 4, 8, 0.125,
              FAKE, None, FAKE, nb, None) == UNSUPPORTED


def test_python_calls_refuse_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k: expected"):
        kv.KVCache(torch.zeros(1, 8, 1, 64, dtype=torch.float16), torch.zeros(1, 8, 1, 64, dtype=torch.float16))
    plan = kv.KVPlan.empty(2, 4, device="cpu")
    with pytest.raises(ValueError, match="ctx_len: expected"):
        kv.kv_plan(i, i, i.reshape(2, 1), i, 16, 4, plan=plan, stream=0)
    with pytest.raises(ValueError, match="parents"):
        kv.ancestor_masks([-1, 1], device="cpu")


def test_ancestor_masks():
    assert kv.ancestor_masks([-1, 0, 0, 1, -1], device="cpu").tolist() == [[1], [3], [5], [11], [16]]
    m = kv.ancestor_masks(list(range(-1, 69)), device="cpu")
    assert m.shape == (70, 2) and m[69].tolist() == [-1, 63] and m[63].tolist() == [-1, 0]
    assert kv.ancestor_masks([], device="cpu").shape == (0, 1)
