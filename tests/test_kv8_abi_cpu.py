"""Host-side refusals of the 8-bit cache's, the rotation's and the sampling's calls (no GPU needed)."""

import ctypes

import pytest
import torch

from ternary_weight_linear_block_gb300 import binding as B
from ternary_weight_linear_block_gb300 import build as BUILD
from ternary_weight_linear_block_gb300 import kv
from tests.test_kv_abi_cpu import cache as cache16

FAKE = 1 << 20          # an aligned, never dereferenced address
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.ensure_built()
    return B.lib()


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=4, page_size=16, heads=2, dim=64, page_stride=2048,
             token_stride=128, head_stride=64, scale_page_stride=32, scale_head_stride=16, dtype=2)
    d.update(kw)
    return B.KVCache8Desc(*(d[n] for n, _ in B.KVCache8Desc._fields_))


def rows(**kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_token_stride=256, q_head_stride=64, k_token_stride=128,
             k_head_stride=64, v_token_stride=128, v_head_stride=64, T=3, Hq=4, slots=FAKE, positions=FAKE, axes=1,
             position_stride=3, turns=FAKE, axis=None, rot=64, q_norm=FAKE, k_norm=FAKE, neighbours=0, dtype=0,
             norm_f32=0, eps=1e-6)
    d.update(kw)
    return B.KVRows(*(d[n] for n, _ in B.KVRows._fields_))


BAD_CACHES = [(dict(dtype=0), INVALID), (dict(dtype=4), INVALID), (dict(k=None), INVALID), (dict(v_scale=None), INVALID),
              (dict(k=FAKE + 8), ALIGN), (dict(k_scale=FAKE + 4), ALIGN), (dict(pages=0), SHAPE),
              (dict(pages=1 << 31), SHAPE), (dict(page_size=4), SHAPE), (dict(page_size=24), SHAPE),
              (dict(page_size=512), SHAPE), (dict(dim=96), SHAPE), (dict(heads=0), SHAPE),
              (dict(page_stride=2040), ALIGN), (dict(token_stride=0), ALIGN), (dict(head_stride=1 << 39), ALIGN),
              (dict(scale_page_stride=30), ALIGN), (dict(scale_head_stride=0), ALIGN)]


def st(fn, *args):
    return getattr(B.lib(), fn)(*args)


def at(x):
    return None if x is None else ctypes.addressof(x)


def test_rotate_write_arguments():
    def w(c8=None, r=None, c16=None):
        return st("tern_kv_rotate_write", at(c16), at(c8), at(r), None)
    assert w(cache(), None) == INVALID and w(None, rows()) == INVALID
    assert w(cache(), rows(), cache16()) == INVALID                     # one cache of the two
    assert w(None, rows(dtype=1), cache16()) == INVALID                 # of the rows' type
    for bad, want in BAD_CACHES:
        assert w(cache(**bad), rows()) == want, bad
    for bad, want in [(dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(rot=-16), INVALID), (dict(dtype=2), INVALID),
                      (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(T=1 << 31), SHAPE),
                      (dict(Hq=65536), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(axes=0), SHAPE),
                      (dict(axes=17), SHAPE), (dict(axes=2, position_stride=2), SHAPE), (dict(T=0), OK),
                      (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
                      (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(positions=None), INVALID),
                      (dict(turns=None), INVALID), (dict(k=FAKE + 8), ALIGN), (dict(q_out=FAKE + 8), ALIGN),
                      (dict(k_norm=FAKE + 4), ALIGN), (dict(v_token_stride=100), ALIGN), (dict(q_head_stride=0), ALIGN)]:
        assert w(cache(), rows(**bad)) == want, bad
    if not torch.cuda.is_available():
        assert w(cache(), rows()) == UNSUPPORTED and w(None, rows(), cache16()) == UNSUPPORTED
        assert w(cache(), rows(Hq=0, q=None, q_out=None, rot=0, positions=None, turns=None)) == UNSUPPORTED


def test_read_arguments():
    def r(c=None, slots=FAKE, t=3, k=FAKE, v=FAKE, dtype=0):
        return st("tern_kv8_read", at(c or cache()), slots, t, k, v, dtype, None)
    for bad, want in BAD_CACHES:
        assert r(cache(**bad)) == want, bad
    for bad, want in [(dict(t=-1), INVALID), (dict(dtype=2), INVALID), (dict(t=1 << 31), SHAPE), (dict(t=0), OK),
                      (dict(slots=None), INVALID), (dict(k=None), INVALID), (dict(v=FAKE + 8), ALIGN)]:
        assert r(**bad) == want, bad


def test_commit_arguments():
    def c(caches=(cache(),), layers=None, b=2, table=FAKE, stride=8, width=8, ctx=FAKE, path=FAKE, pw=4, plen=FAKE,
          out=FAKE + 64):
        array = (B.KVCache8Desc * len(caches))(*caches)
        return st("tern_kv8_commit", ctypes.addressof(array), len(caches) if layers is None else layers, table, stride,
                  width, ctx, path, pw, plen, out, b, None)
    for bad, want in BAD_CACHES:
        assert c((cache(), cache(**bad))) == want, bad
    assert c((cache(), cache(pages=5))) == SHAPE and c((cache(), cache(scale_head_stride=32))) == SHAPE
    assert c(layers=0) == INVALID and c(b=-1) == INVALID and c(pw=-1) == INVALID
    assert c(b=0) == OK and c(b=65536) == SHAPE and c(pw=257) == SHAPE and c(stride=4) == SHAPE
    assert c(ctx=None) == INVALID and c(path=None) == INVALID and c(plen=None) == INVALID
    assert c(out=None) == INVALID and c(out=FAKE) == INVALID and c(table=None) == INVALID


@pytest.mark.parametrize("new,hq", [(1, 4), (8, 4), (64, 4)])      # the kernels of few rows and of many
def test_attention_arguments(new, hq):
    need = B.tern_tree_attention8_workspace_bytes(new, hq, 2, 64)
    assert need > B.TERN_TREE_ATTENTION_ZERO_BYTES

    def a(c=None, q=FAKE, qs=(256, 64), dtype=0, table=FAKE, stride=8, width=8, ctx=FAKE, start=FAKE, mask=FAKE,
          words=1, b=2, t=9, hq=hq, new=new, scale=0.125, out=FAKE, lse=None, ws=FAKE, nb=need):
        return st("tern_tree_attention8", q, *qs, dtype, at(c or cache()), table, stride, width, ctx, start, mask,
                  words, b, t, hq, new, scale, out, lse, ws, nb, None)
    for bad, want in BAD_CACHES:
        assert a(cache(**bad)) == want, bad
    for bad, want in [(dict(b=-1), INVALID), (dict(t=-1), INVALID), (dict(words=-1), INVALID), (dict(dtype=2), INVALID),
                      (dict(new=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
                      (dict(hq=0), SHAPE), (dict(hq=5), SHAPE), (dict(b=65537), SHAPE), (dict(new=257), SHAPE),
                      (dict(words=5), SHAPE), (dict(stride=4), SHAPE), (dict(t=1 << 27), SHAPE), (dict(q=None), INVALID),
                      (dict(ctx=None), INVALID), (dict(start=None), INVALID), (dict(out=None), INVALID),
                      (dict(table=None), INVALID), (dict(words=0), INVALID), (dict(q=FAKE + 8), ALIGN),
                      (dict(out=FAKE + 8), ALIGN), (dict(qs=(250, 64)), ALIGN), (dict(ws=None), WORKSPACE),
                      (dict(nb=need - 1), WORKSPACE), (dict(ws=FAKE + 8), ALIGN), (dict(b=0), OK), (dict(t=0), OK),
                      (dict(new=0), OK)]:
        assert a(**bad) == want, bad


def test_workspace_sizes():
    ask = B.tern_tree_attention8_workspace_bytes
    for bad in [(0, 4, 2, 64), (257, 4, 2, 64), (1, 4, 0, 64), (1, 3, 2, 64), (1, 1, 2, 64), (1, 4, 2, 96)]:
        assert ask(*bad) == 0, bad
    assert ask(1, 4, 4, 64) < ask(16, 4, 4, 64) < ask(256, 8, 2, 64)


def test_sample_arguments():
    def s(x=FAKE, stride=100, rows=3, vocab=100, dtype=0, u=FAKE, token=FAKE):
        return st("tern_sample", x, stride, rows, vocab, dtype, u, None, None, None, None, token, None)
    for bad, want in [(dict(rows=-1), INVALID), (dict(dtype=-1), INVALID), (dict(dtype=3), INVALID),
                      (dict(vocab=0), SHAPE), (dict(vocab=2 ** 18 + 1, stride=2 ** 19), SHAPE), (dict(rows=1 << 20), SHAPE),
                      (dict(stride=99), SHAPE), (dict(stride=1 << 39), SHAPE), (dict(rows=0), OK), (dict(x=None), INVALID),
                      (dict(u=None), INVALID), (dict(token=None), INVALID), (dict(x=FAKE + 1), ALIGN),
                      (dict(x=FAKE + 2, dtype=2), ALIGN)]:
        assert s(**bad) == want, bad
    if not torch.cuda.is_available():
        assert s(x=FAKE + 2) == UNSUPPORTED


def test_accept_arguments():
    def a(tokens=FAKE, target=FAKE, parent=FAKE, start=FAKE, b=2, t=9, width=4, path=FAKE, plen=FAKE, nxt=FAKE):
        return st("tern_tree_accept", tokens, target, parent, start, b, t, width, path, plen, nxt, None)
    for bad, want in [(dict(b=-1), INVALID), (dict(t=-1), INVALID), (dict(b=65537), SHAPE), (dict(t=1 << 31), SHAPE),
                      (dict(width=0), SHAPE), (dict(width=257), SHAPE), (dict(b=0), OK), (dict(start=None), INVALID),
                      (dict(path=None), INVALID), (dict(plen=None), INVALID), (dict(nxt=None), INVALID),
                      (dict(tokens=None), INVALID), (dict(target=None), INVALID), (dict(parent=None), INVALID)]:
        assert a(**bad) == want, bad


def test_rotary():
    r = kv.Rotary([1.0] * 8 + [0.5, -0.25] * 4, device="cpu")
    turn = [t % 2 ** 64 for t in r.turns.tolist()]
    # 1 / (2 pi) of a turn, to the last bit; half of it, and a quarter the other way
    assert turn[0] == 2935890503282001226 and abs(turn[8] - turn[0] / 2) <= 1
    assert (turn[9] + turn[0] // 4) % 2 ** 64 <= 1 or 2 ** 64 - (turn[9] + turn[0] // 4) % 2 ** 64 <= 1
    assert r.rot == 32 and r.axes == 1 and kv.Rotary.geometric(64, device="cpu").rot == 64
    assert kv.Rotary([1.0] * 8, axis=[0, 2, 1] * 2 + [0, 0], device="cpu").axes == 3
    for bad in (dict(freq=[1.0] * 7), dict(freq=[]), dict(freq=[float("nan")] * 8), dict(freq=[1.0] * 8, axis=[0] * 7),
                dict(freq=[1.0] * 8, axis=[-1] * 8)):
        with pytest.raises(ValueError, match="freq|axis"):
            kv.Rotary(**bad, device="cpu")


def test_python_calls_refuse_host_tensors():
    x = torch.zeros(1, 8, 1, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="k: expected"):
        kv.KVCache8(x, x, torch.zeros(1, 1, 8), torch.zeros(1, 1, 8))
