"""Plain statements of the 8-bit cache, the rotation, sampling and acceptance, for the tests (host only)."""

import math

import numpy as np
import torch

LARGEST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def quantise(x, kind):
    """Rows (float32, last axis) as codes and units, in the operator's own float32 steps."""
    most = x.abs().amax(-1, keepdim=True)
    nan = torch.isnan(x).any(-1, keepdim=True)
    whole = torch.isfinite(most) & ~nan
    some = whole & (most >= 2.0 ** -100)
    # (a number divided by a tensor is a product with its reciprocal, two roundings)
    largest = torch.full_like(most, LARGEST[kind])
    y = torch.where(some, x * (largest / torch.where(some, most, torch.ones(()))), torch.zeros(()))
    codes = y.round().to(torch.int8) if kind == torch.int8 else y.to(kind)
    unit = torch.where(some, most / largest, torch.where(whole, torch.zeros(()), torch.full((), math.nan)))
    return codes, unit[..., 0]


def rotate(x, norm, eps, freq, axis, positions, neighbours):
    """Rows [T, H, D] (float64) normalised and turned; positions [axes, T]."""
    x = x.double()
    if norm is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * norm.double()
    half = len(freq)
    if half == 0:
        return x
    y = x.clone()
    for j in range(half):
        p = positions[axis[j] if axis is not None else 0].tolist()
        # the angle's part of a turn in whole numbers: positions may be of any size
        angle = torch.tensor([math.fmod(t * freq[j], 2 * math.pi) for t in p], dtype=torch.float64)
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = (2 * j, 2 * j + 1) if neighbours else (j, j + half)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def sample(x, u, temperature, top_k, top_p, min_p):
    """(token, weights of the kept ones, their running sum by index) of one row, in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    n, most = len(x), x.max()
    if most == -np.inf:
        return -1, None, None
    order = np.lexsort((np.arange(n), -x))
    if not temperature > 0 or top_k == 1 or top_p <= 0:
        w = np.zeros(n)
        w[order[0]] = 1
        return int(order[0]), w, np.cumsum(w)
    with np.errstate(all="ignore"):
        w = np.where(x == most, 1.0, np.exp((x - most) / temperature))
    w = np.where(np.isnan(w), 0.0, w)[order]
    if 0 < top_k < n:
        w[top_k:] = 0
    if min_p > 0:
        w[w < min(min_p, 1.0)] = 0
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        w[before >= top_p * w.sum()] = 0
    kept = np.zeros(n)
    kept[order] = w
    run = np.cumsum(kept)
    return int((run <= u * run[-1]).sum()), kept, run


def accept(tokens, target, parents, starts, width):
    path, length, following = [], [], []
    for b in range(len(starts) - 1):
        n = min(starts[b + 1] - starts[b], width)
        t, g, p = (x[starts[b]:starts[b] + n] for x in (tokens, target, parents))
        at, nxt = ([0], g[0]) if n > 0 else ([], -1)
        while at:
            fits = [j for j in range(at[-1] + 1, n) if p[j] == at[-1] and t[j] == nxt]
            if not fits:
                break
            at.append(fits[0])
            nxt = g[fits[0]]
        path.append(at + [-1] * (width - len(at)))
        length.append(len(at))
        following.append(nxt)
    return path, length, following
