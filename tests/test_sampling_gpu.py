"""Sampling and the acceptance of drafts against plain statements of them."""

import numpy as np
import pytest
import torch

from ternary_weight_linear_block_gb300 import sampling
from tests import kv8_reference as R
from tests.gpu_helpers import ensure_lib, poison

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def dev(x, dtype=F32):
    return None if x is None else torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def check(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Weights are off by 2^-28 at most, so running sums by 2^-28 of the whole and the border of top-p
    by one token: a token is right where u times the sum is inside its own part, widened by 2^-26 of the sum
    (and where the set of kept ones is the statement's for top_p off by that much)."""
    rows = x.shape[0]
    got = sampling.sample(x, dev(u), dev(temperature), dev(top_k, torch.int32), dev(top_p), dev(min_p)).tolist()
    values = x.float().cpu().numpy()
    f32 = np.float32
    for r in range(rows):
        t = 1.0 if temperature is None else float(f32(temperature[r]))
        k = 0 if top_k is None else int(top_k[r])
        p = 1.0 if top_p is None else float(f32(top_p[r]))
        m = 0.0 if min_p is None else float(f32(min_p[r]))
        want, kept, run = R.sample(values[r], float(f32(u[r])), t, k, p, m)
        if got[r] == want:
            continue
        # the same filter moved by what the weights' errors can move it
        near = []
        for q in ([p] if p >= 1 else [p * (1 - 2.0 ** -26), min(p * (1 + 2.0 ** -26), 1 - 2.0 ** -30)]):
            _, kept, run = R.sample(values[r], float(f32(u[r])), t, k, q, m)
            i, goal, slack = got[r], float(f32(u[r])) * run[-1], run[-1] * 2.0 ** -26
            near.append(0 <= i < len(run) and kept[i] > 0 and run[i] - kept[i] - slack <= goal < run[i] + slack)
        assert any(near), (r, got[r], want, t, k, p, m)


def logits(rng, rows, vocab, dtype, likely=20):
    x = 2 * rng.standard_normal((rows, vocab)).astype(np.float32)
    for r in range(rows):
        at = rng.integers(0, vocab, likely)
        x[r, at] += rng.uniform(6, 18) * rng.random(likely)
    return torch.from_numpy(x).to(dtype).cuda()


def filters(rng, rows, names):
    return {"temperature": rng.uniform(0.5, 1.5, rows) if "t" in names else None,
            "top_k": rng.integers(1, 100, rows) if "k" in names else None,
            "top_p": rng.uniform(0.3, 0.999, rows) if "p" in names else None,
            "min_p": rng.uniform(0.001, 0.2, rows) if "m" in names else None}


@pytest.mark.parametrize("names", ["", "t", "tk", "tp", "tm", "tkp", "tkpm"])
@pytest.mark.parametrize("rows,vocab,dtype", [
    (1, 1, F32), (2, 2, BF), (3, 7, HF), (5, 31, F32), (4, 1000, BF), (3, 4096, F32), (9, 50001, HF), (2, 131072, BF),
    (1, 262144, F32), (40, 20000, BF), (170, 3001, F32), (400, 999, HF)])
def test_sample(rows, vocab, dtype, names):
    rng = np.random.default_rng(rows * 7 + vocab)
    check(logits(rng, rows, vocab, dtype), rng.random(rows), **filters(rng, rows, names))


@pytest.mark.parametrize("rows,vocab,dtype,names", [
    (310, 33001, F32, "tp"), (120, 70001, HF, "tkp"), (307, 128257, BF, "tp")])
def test_more_rows_than_fit(rows, vocab, dtype, names):
    """Long rows that several CTAs share although not all of them run at once."""
    rng = np.random.default_rng(rows + vocab)
    check(logits(rng, rows, vocab, dtype), rng.random(rows), **filters(rng, rows, names))


@pytest.mark.parametrize("rows,vocab", [(3, 150001), (30, 40000), (200, 5000)])
def test_filters_that_keep_many(rows, vocab):
    """Borders beyond the short list: searched by histograms."""
    rng = np.random.default_rng(vocab)
    for dtype in (BF, F32):
        x = logits(rng, rows, vocab, dtype, likely=1)
        u = rng.random(rows)
        check(x, u, top_k=rng.integers(385, vocab, rows))
        check(x, u, top_p=rng.uniform(0.6, 0.9999, rows), temperature=np.full(rows, 1.3))
        check(x, u, top_k=rng.integers(385, vocab, rows), top_p=rng.uniform(0.5, 0.99, rows), min_p=np.full(rows, 1e-6))
        check(x, u, top_k=np.full(rows, vocab), temperature=np.full(rows, 40.0), top_p=np.full(rows, 0.5))


@pytest.mark.parametrize("vocab", [100, 5000, 262144])
def test_ties(vocab):
    """Few distinct logits: the lowest indices of the border's are kept."""
    rng = np.random.default_rng(vocab)
    for dtype in (BF, HF, F32):
        x = torch.from_numpy(rng.integers(0, 3, (6, vocab)).astype(np.float32)).to(dtype).cuda()
        x[0] = 0
        x[1] = -0.0
        x[1, ::2] = 0.0
        x[2] = 7
        for k in (1, 2, 50, 90):
            check(x, [0.0, 0.3, 0.5, 0.7, 0.9, 1 - 2.0 ** -24], top_k=[k] * 6)
        check(x, rng.random(6), top_p=[0.001, 0.5, 0.25, 0.9, 0.99, 0.1])
        check(x, rng.random(6), top_p=[0.001, 0.5, 0.25, 0.9, 0.99, 0.1], top_k=[70, 3, 99, 10, 50, 60])
        check(x, rng.random(6), min_p=[1.0, 1.0, 1.0, 1.0, 0.5, 0.2])


def test_the_largest():
    rng = np.random.default_rng(3)
    x = logits(rng, 7, 70000, BF)
    x[2] = 1
    x[3, 5], x[3, 9], x[4, 69999] = 90, 90, 95
    want = [int(r.argmax()) if i != 2 else 0 for i, r in enumerate(x.float().cpu().numpy())]
    assert want[3] == 5 and want[4] == 69999
    u = dev(rng.random(7))
    for kw in ({"temperature": dev([0.0, -1.0, 0, 0, float("nan"), 0, 1e-30])},
               {"top_k": dev([1] * 7, torch.int32)}, {"top_p": dev([0.0, -1.0, 0, 0, 1e-30, 1e-9, 0])}):
        assert sampling.sample(x, u, **kw).tolist() == want


def test_values_that_are_not_ordinary():
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(8, 40, device="cuda")
    x[0] = -inf
    x[1] = nan
    x[2, 3:] = -inf
    x[3, 1:] = nan
    x[4, 7], x[4, 30] = inf, inf
    x[5], x[5, 11] = -inf, -3e38
    x[6, :20] = 3e38
    x[7, 0], x[7, 1:] = nan, -inf
    u = [0.9, 0.9, 0.9, 0.9, 0.9, 0.9, 0.01, 0.5]
    for dtype in (F32, BF):
        y = x.to(dtype)
        for kw in ({}, {"top_p": [0.9] * 8}, {"top_k": [30] * 8}, {"min_p": [0.5] * 8},
                   {"temperature": [inf] * 8}, {"temperature": [1e-38] * 8}):
            got = sampling.sample(y, dev(u), **{k: dev(v, torch.int32 if k == "top_k" else F32) for k, v in kw.items()})
            got = got.tolist()
            assert got[0] == got[1] == got[7] == -1 and got[2] == (1 if kw.get("top_p") == [0.5] * 8 else 2), (kw, got)
            assert got[3] == 0 and got[4] == 30 and got[5] == 11 and 0 <= got[6] < 20, (kw, got)
    # random numbers outside their range
    z = torch.zeros(4, 10, device="cuda")
    assert sampling.sample(z, dev([-1.0, 1.0, nan, 2.0])).tolist() == [0, 9, 0, 9]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_rows_anywhere(dtype, shift):
    """Rows at every alignment, with what stands before and behind them large: it is not theirs."""
    rng = np.random.default_rng(shift)
    whole = torch.full((5, 3007), 1e4, dtype=dtype, device="cuda")
    x = whole[:, shift:shift + 2999]
    x.copy_(logits(rng, 5, 2999, dtype))
    check(x, rng.random(5))
    check(x, rng.random(5), top_k=[5] * 5, top_p=[0.9] * 5)
    check(x[2:3], rng.random(1), top_p=[0.99])


def test_out_stream_and_no_rows():
    rng = np.random.default_rng(4)
    x, u = logits(rng, 12, 30011, BF), dev(rng.random(12))
    want = sampling.sample(x, u)
    out = poison(torch.empty(14, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sampling.sample(x, u, out=out[:12], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(out[:12], want) and (out[12:].view(torch.uint8) == 255).all()
    assert torch.equal(sampling.sample(x, u, stream=side), want)
    assert sampling.sample(x[:0], u[:0]).shape == (0,)


def test_captured_and_replayed():
    rng = np.random.default_rng(5)
    x, u, k = logits(rng, 3, 60000, BF), dev(rng.random(3)), dev([40, 500, 1], torch.int32)
    out = torch.empty(3, dtype=torch.int32, device="cuda")
    sampling.sample(x, u, top_k=k, out=out)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sampling.sample(x, u, top_k=k, out=out)
    for seed in range(4):
        u.copy_(dev(np.random.default_rng(seed).random(3)))
        x.copy_(x.roll(997, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sampling.sample(x, u, top_k=k))


def test_sample_refusals():
    x, u = torch.zeros(3, 8, device="cuda"), torch.zeros(3, device="cuda")
    for what, call in [("logits", lambda: sampling.sample(x.double(), u)),
                       ("logits", lambda: sampling.sample(x.t(), torch.zeros(8, device="cuda"))),
                       ("logits", lambda: sampling.sample(x[0], u)), ("u: expected", lambda: sampling.sample(x, u.half())),
                       ("one number each row", lambda: sampling.sample(x, u[:2])),
                       ("top_k", lambda: sampling.sample(x, u, top_k=u)),
                       ("one number each row", lambda: sampling.sample(x, u, top_p=u[:1])),
                       ("token", lambda: sampling.sample(x, u, out=u))]:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(sampling.B.TernError):
        sampling.sample(torch.zeros(1, 2 ** 18 + 1, device="cuda"), u[:1])


def make_trees(rng, sizes, words):
    tokens, target, parents, starts = [], [], [], [0]
    for n in sizes:
        p = [-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)]
        tokens += rng.integers(0, words, n).tolist()
        target += rng.integers(0, words, n).tolist()
        parents += p[:n]
        starts.append(starts[-1] + n)
    return tokens, target, parents, starts


@pytest.mark.parametrize("sizes,words", [
    ([1], 3), ([0], 3), ([7, 0, 1, 33], 2), ([256, 31, 32], 2), ([64, 65, 100], 1), ([5] * 300, 3), ([200], 4)])
def test_accept(sizes, words):
    rng = np.random.default_rng(len(sizes) + words)
    tokens, target, parents, starts = make_trees(rng, sizes, words)
    width = max(sizes + [1])
    for w in {width, max(1, width // 2)}:
        got = sampling.accept(dev(tokens, torch.int32), dev(target, torch.int32), dev(parents, torch.int32),
                              dev(starts, torch.int32), w)
        want = R.accept(tokens, target, parents, starts, w)
        for g, x in zip(got, want):
            assert g.tolist() == x


def test_accept_long_chains_and_bad_parents():
    n = 256
    chain = list(range(-1, n - 1))
    tokens = [i % 9 for i in range(n)]
    target = [(i + 1) % 9 for i in range(n)]
    i32 = torch.int32
    path, length, following = sampling.accept(dev(tokens, i32), dev(target, i32), dev(chain, i32), dev([0, n], i32), n)
    assert length.tolist() == [n] and path[0].tolist() == list(range(n)) and following.tolist() == [n % 9]
    bad = [5, 0, 2, 7, -1, 1 << 30, -(1 << 31), 1] + chain[8:]
    same = [0] * n
    path, length, following = sampling.accept(dev(same, i32), dev(same, i32), dev(bad, i32), dev([0, n], i32), n)
    assert path[0].tolist()[:length] == R.accept(same, same, bad, [0, n], n)[0][0][:int(length)]
    # row starts that are none: nothing is read
    out = sampling.accept(dev([1, 2], i32), dev([1, 2], i32), dev([-1, 0], i32), dev([-4, 1, 9, 1], i32), 3)
    assert out[1].tolist() == [0, 0, 0] and out[2].tolist() == [-1] * 3 and (out[0] == -1).all()


def test_accept_refusals():
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    for what, call in [("tokens", lambda: sampling.accept(i.float(), i, i, i, 2)),
                       ("one each token", lambda: sampling.accept(i, i[:1], i, i, 2)),
                       ("path", lambda: sampling.accept(i, i, i, i, 2, path=torch.zeros(1, 3, dtype=torch.int32,
                                                                                   device="cuda"))),
                       ("row each request", lambda: sampling.accept(i, i, i, i, 2, path_len=i))]:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(sampling.B.TernError):
        sampling.accept(i, i, i, i, 257)
