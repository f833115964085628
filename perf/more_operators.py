"""An 8-bit key/value cache, rotated rows, sampling and acceptance of drafts: the cases that are measured.

Five operators, which a step of decoding or of verifying drafts uses around the paged cache:

* ``rotate``: norms of queries and keys for each head and their rotary positions (one axis or several), with the keys
  and values written to the cache's slots in the same pass, as 16-bit values or in 8 bits;
* ``store``: keys and values quantised as they are written to an 8-bit cache, and read back from their slots;
* ``attn``: attention of every request's tree of drafted tokens over an 8-bit cache;
* ``sample``: tokens from logits with temperature, top-k, top-p and min-p, from given random numbers;
* ``accept``: the path of each tree of drafts that agrees with the sampled tokens.

``run`` is the plain form (32-bit torch operations, 64-bit ones for angles and for sampling's sums, rounded once) or,
where ``own`` is true, the calls that a user makes of the framework.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST = {"int8": 127.0, "e4m3": 448.0}
SMALLEST = 2.0 ** -100                # rows of no value above this are stored as zeros


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the 16 rows of one decode step of the 5120-wide model, 16-bit cache: the smallest call, latency counts
        dict(name="rotate decode", op="rotate", requests=2, new=8, ctx=1000, page=16, kv_heads=20, group=2, dim=128,
             dtype="bf16", cache="bf16", rot=128, axes=1, neighbours=False, norm=True),
        # a prompt with images: positions in time, height and width, a quarter of the head rotated, 8-bit cache
        dict(name="rotate images", op="rotate", requests=5, new=9001, ctx=77, page=64, kv_heads=4, group=6, dim=256,
             dtype="bf16", cache="e4m3", rot=64, axes=3, neighbours=False, norm=True),
        # one decode step's rows into an int8 cache
        dict(name="store decode", op="store", requests=2, new=8, ctx=1000, page=16, kv_heads=20, group=2, dim=128,
             dtype="bf16", cache="int8"),
        # a prompt pass: 65521 tokens at most, 8 key heads
        dict(name="store prompts", op="store", requests=13, new=9001, ctx=77, page=64, kv_heads=8, group=4, dim=128,
             dtype="fp16", cache="int8"),
        # 16 requests of one token each at short contexts: latency counts
        dict(name="attn one token", op="attn", requests=16, new=1, ctx=700, page=16, kv_heads=20, group=2, dim=128,
             dtype="bf16", cache="int8"),
        # ordinary serving: 64 requests of one token at uneven contexts
        dict(name="attn batch", op="attn", requests=64, new=1, ctx=16001, page=16, kv_heads=8, group=4, dim=128,
             dtype="bf16", cache="int8"),
        # one long conversation, a tree of four drafts, head size 256
        dict(name="attn long", op="attn", requests=1, new=4, ctx=131001, page=64, kv_heads=4, group=6, dim=256,
             dtype="fp16", cache="e4m3"),
        # wide trees: many rows on each key head, the most arithmetic for each byte
        dict(name="attn wide tree", op="attn", requests=4, new=29, ctx=20003, page=32, kv_heads=8, group=4, dim=128,
             dtype="bf16", cache="int8"),
        # the tokens of a small decode step, every filter in use
        dict(name="sample decode", op="sample", rows=4, vocab=131072, dtype="bf16", filters="all"),
        # verification of drafts for many requests: a row each, filters as the requests ask, an odd vocabulary
        dict(name="sample batch", op="sample", rows=250, vocab=250007, dtype="bf16", filters="mixed"),
        # 16 requests of up to 16 drafts
        dict(name="accept decode", op="accept", requests=16, new=16),
        # a thousand requests with wide trees
        dict(name="accept batch", op="accept", requests=1000, new=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "store", "attn", "attn", "attn", "sample", "sample", "accept"])
    if op == "accept":
        requests = _log(rng, 1, 1000)
        return dict(op=op, requests=requests, new=_log(rng, 1, 64))
    if op == "sample":
        vocab = _log(rng, 1000, 262144)
        return dict(op=op, rows=_log(rng, 1, max(1, min(300, 60000000 // vocab))), vocab=vocab,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    filters=rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]))
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 20])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    case = dict(op=op, page=rng.choice([16, 32, 64, 128]), kv_heads=kv_heads, group=group, dim=dim,
                dtype=rng.choice(["bf16", "fp16"]), cache=rng.choice(["int8", "e4m3"]))
    row = kv_heads * dim
    if op == "store":
        requests = _log(rng, 1, 64)
        return dict(case, requests=requests, new=_log(rng, 1, max(1, 60000000 // (row * requests))),
                    ctx=_log(rng, 1, 300))
    if op == "rotate":
        requests = _log(rng, 1, 64)
        rot = rng.choice([r for r in (16, 32, 64, 80, 128, 256) if r <= dim])
        most = max(1, 150000000 // (row * (group + 2) * requests))
        return dict(case, requests=requests, new=_log(rng, 1, most), ctx=_log(rng, 1, 200000 // requests),
                    cache=rng.choice([case["dtype"], "int8", "e4m3"]), rot=rot, axes=rng.choice([1, 1, 2, 3]),
                    neighbours=rng.random() < 0.3, norm=rng.random() < 0.7)
    requests = _log(rng, 1, 128)
    new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 40)])
    # at most the batch's keys and the wide tree's arithmetic
    most = min(1.3e8 * 4 / (requests * row), 8.0e9 / (requests * new * group * row), 131072)
    return dict(case, requests=requests, new=new, ctx=_log(rng, 1, max(1, most)))


def _lengths(case):
    """Cached and new tokens of every request: uneven, by the case alone, the largest as the case says."""
    rng = random.Random("%(op)s %(requests)d %(new)d" % case)
    most = case.get("ctx", 1)
    ctx = [max(1, int(most * rng.uniform(0.25, 1.0))) for _ in range(case["requests"])]
    new = [max(1, int(math.ceil(case["new"] * rng.uniform(0.5, 1.0)))) for _ in range(case["requests"])]
    ctx[-1], new[-1] = most, case["new"]
    return ctx, new


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ inputs

def _signed(word):
    return word - (1 << 64) if word >= 1 << 63 else word


def _tree(n, key):
    """A drafted tree: parent of each token (-1: the context), and each token's ancestors as bits."""
    rng, bits = random.Random(key), []
    parent = [-1] + [rng.randrange(max(0, i - 6), i) for i in range(1, n)]
    for i, p in enumerate(parent):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return parent, bits


def _prepare_sample(case, gen, dev):
    rows, vocab, filters = case["rows"], case["vocab"], case["filters"]

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(rows, generator=gen, device=dev)

    # a wide bulk and a few likely tokens a row, as a trained model's logits have; some rows are sure, some open
    logits = torch.randn(rows, vocab, generator=gen, device=dev) * 2
    likely = torch.randint(vocab, (rows, 40), generator=gen, device=dev)
    logits.scatter_add_(1, likely, uniform(8, 18)[:, None] * torch.rand(rows, 40, generator=gen, device=dev))
    s = dict(case=case, logits=logits.to(TYPES[case["dtype"]]), u=torch.rand(rows, generator=gen, device=dev),
             temperature=uniform(0.6, 1.3), top_k=None, top_p=None, min_p=None)
    if filters in ("top_k", "all", "mixed"):
        s["top_k"] = torch.randint(1, 100, (rows,), generator=gen, device=dev).to(torch.int32)
    if filters in ("top_p", "all", "mixed"):
        s["top_p"] = uniform(0.7, 0.99)
    if filters in ("min_p", "all", "mixed"):
        s["min_p"] = uniform(0.01, 0.1)
    if filters == "mixed":
        # each request asks for some of them; some are greedy
        off = torch.rand(4, rows, generator=gen, device=dev) < torch.tensor([[0.5], [0.4], [0.6], [0.1]], device=dev)
        s["top_k"] = torch.where(off[0], 0, s["top_k"]).to(torch.int32)
        s["top_p"] = torch.where(off[1], 1.0, s["top_p"])
        s["min_p"] = torch.where(off[2], 0.0, s["min_p"])
        s["temperature"] = torch.where(off[3], 0.0, s["temperature"])
    return s


def _prepare_accept(case, seed, dev):
    rng = random.Random(seed)
    _, new = _lengths(case)
    parents, tokens, target, starts = [], [], [], [0]
    for n in new:
        parent, _ = _tree(n, rng.random())
        token = [rng.randrange(100000) for _ in range(n)]
        for i in range(2, n):
            if rng.random() < 0.05:                              # a draft that another draft has too
                token[i] = token[rng.randrange(1, i)]
        children = [[] for _ in range(n)]
        for i in range(1, n):
            children[parent[i]].append(i)
        parents += parent
        tokens += token
        # three of four sampled tokens are one of the drafts that follow
        target += [token[rng.choice(c)] if c and rng.random() < 0.75 else rng.randrange(100000) for c in children]
        starts.append(starts[-1] + n)
    ints = dict(dtype=torch.int32, device=dev)
    return dict(case=case, parents=torch.tensor(parents, **ints), tokens=torch.tensor(tokens, **ints),
                target=torch.tensor(target, **ints), row_start=torch.tensor(starts, **ints), max_new=max(new))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, gen, dev)
    if case["op"] == "accept":
        return _prepare_accept(case, seed, dev)
    ctx, new = _lengths(case)
    page, requests = case["page"], case["requests"]
    total = sum(new)
    int32 = dict(dtype=torch.int32, device=dev)
    needed = [_pages(c + n, page) for c, n in zip(ctx, new)]
    width = max(needed) + 1
    pages = sum(needed) + 8
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    s = dict(case=case, total=total, page=page, pages=pages, max_new=max(new),
             ctx_len=torch.tensor(ctx, **int32), new_len=torch.tensor(new, **int32))
    at = torch.arange(width, device=dev)[None, :]
    first = torch.tensor([0] + needed[:-1], device=dev).cumsum(0)[:, None]
    known = at < torch.tensor(needed, device=dev)[:, None]
    s["table"] = torch.where(known, order[(first + at).clamp(max=pages - 1)], 0).to(torch.int32)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["row_start"] = torch.tensor(starts, **int32)
    dtype, heads, dim, kind = TYPES[case["dtype"]], case["kv_heads"], case["dim"], case["cache"]
    q_heads = heads * case["group"]
    request = torch.repeat_interleave(torch.arange(requests, device=dev), s["new_len"].long())
    s["local"] = torch.arange(total, device=dev) - s["row_start"].long()[request]
    s["request"] = request
    position = s["ctx_len"].long()[request] + s["local"]
    s["slots"] = s["table"][request, position // page].long() * page + position % page

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    # a few channels of large mean, as trained models' keys have
    mean = torch.zeros(heads, dim, device=dev, dtype=dtype)
    mean[:, torch.randperm(dim, generator=gen, device=dev)[:4]] = 3.0
    shape = pages, page, heads, dim
    if kind in CODES:
        for name in ("k", "v"):
            if case["op"] == "attn":
                values = normal(*shape)
                values = values.add_(mean) if name == "k" else values
                values = values.mul_(LARGEST[kind] / 7).clamp_(-LARGEST[kind], LARGEST[kind])
                s[name + "_cache"] = (values.round_() if kind == "int8" else values).to(CODES[kind])
                spread = torch.randn(pages, heads, page, generator=gen, device=dev).mul_(0.2).exp_()
                s[name + "_scale"] = spread * (7 / LARGEST[kind])
            else:
                s[name + "_cache"] = torch.zeros(shape, device=dev, dtype=torch.int8).view(CODES[kind])
                s[name + "_scale"] = torch.zeros(pages, heads, page, device=dev)
    else:
        s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
    # queries, keys and values as the qkv linear leaves them: slices of one row
    qkv = normal(total, (q_heads + 2 * heads) * dim)
    s["q"] = qkv[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    s["k"] = qkv[:, q_heads * dim:(q_heads + heads) * dim].unflatten(1, (heads, dim))
    s["v"] = qkv[:, (q_heads + heads) * dim:].unflatten(1, (heads, dim))
    s["k"].add_(mean)
    if case["op"] == "attn":
        trees = [_tree(n, seed * 1000003 + b) for b, n in enumerate(new)]
        s["mask"] = torch.tensor([[_signed(w)] for _, bits in trees for w in bits], dtype=torch.int64, device=dev)
    if case["op"] == "rotate":
        half, axes = case["rot"] // 2, case["axes"]
        s["freq"] = 1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        s["axis"] = torch.arange(half, device=dev) % axes
        # the rows of an image have places in its height and width too
        at = [position, position // 7 % 96, position % 84][:axes]
        s["positions"] = torch.stack(at).to(torch.int32) if axes > 1 else position.to(torch.int32)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = (1 + 0.1 * torch.randn(dim, generator=gen, device=dev)).to(dtype)
            s["k_norm"] = (1 + 0.1 * torch.randn(dim, generator=gen, device=dev)).to(dtype)
    return s


# ------------------------------------------------------------------ one pass

EPS = 1e-6


def _codes(x, kind):
    """Rows quantised along the last axis: codes, and a scale each."""
    most = x.abs().amax(-1, keepdim=True)
    whole = torch.isfinite(most)
    some = whole & (most >= SMALLEST)
    y = torch.where(some, x * (LARGEST[kind] / torch.where(some, most, 1.0)), 0.0)
    codes = y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    scale = torch.where(some, most / LARGEST[kind], torch.where(whole, 0.0, math.nan))
    return codes, scale[..., 0]


def _plain_write(s, k, v):
    kind, page, slots = s["case"]["cache"], s["page"], s["slots"]
    if kind not in CODES:
        s["k_cache"].flatten(0, 1)[slots] = k.to(s["k_cache"].dtype)
        s["v_cache"].flatten(0, 1)[slots] = v.to(s["v_cache"].dtype)
        return
    (kc, ks), (vc, vs) = _codes(k.float(), kind), _codes(v.float(), kind)
    s["k_cache"].view(torch.int8).flatten(0, 1)[slots] = kc.view(torch.int8)
    s["v_cache"].view(torch.int8).flatten(0, 1)[slots] = vc.view(torch.int8)
    s["k_scale"][slots // page, :, slots % page] = ks
    s["v_scale"][slots // page, :, slots % page] = vs


def _plain_read(s):
    slots, page, dtype = s["slots"], s["page"], TYPES[s["case"]["dtype"]]
    k = s["k_cache"].view(torch.int8).flatten(0, 1)[slots].view(s["k_cache"].dtype).float()
    v = s["v_cache"].view(torch.int8).flatten(0, 1)[slots].view(s["v_cache"].dtype).float()
    k = k * s["k_scale"][slots // page, :, slots % page, None]
    v = v * s["v_scale"][slots // page, :, slots % page, None]
    return k.to(dtype), v.to(dtype)


def _plain_store(s):
    _plain_write(s, s["k"], s["v"])
    return _plain_read(s)


def _plain_rotate(s):
    case, dim, rot = s["case"], s["case"]["dim"], s["case"]["rot"]
    at = s["positions"].double()
    at = at[s["axis"]].T if case["axes"] > 1 else at[:, None]
    angle = at * s["freq"]                                                  # [T, rot / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["neighbours"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        c, d = a * cos - b * sin, b * cos + a * sin
        pair = torch.stack([c, d], -1).flatten(-2) if case["neighbours"] else torch.cat([c, d], -1)
        return torch.cat([pair, x[..., rot:]], -1)

    q = turned(s["q"], s["q_norm"]).to(s["q"].dtype)
    _plain_write(s, turned(s["k"], s["k_norm"]), s["v"])
    return (q,) + (_plain_read(s) if case["cache"] in CODES else (s["k_cache"], s["v_cache"]))


def _plain_attn(s):
    case, table, q, page = s["case"], s["table"].long(), s["q"], s["page"]
    dev, dim, group = q.device, case["dim"], case["group"]
    starts, ctx, width = s["row_start"].long(), s["ctx_len"].long(), s["max_new"]
    new = starts[1:] - starts[:-1]
    keys = table.shape[1] * page

    def gathered(codes, scale):                                             # [B, L, H, D]
        x = codes.view(torch.int8)[table].view(codes.dtype).float()
        return x.mul_(scale[table].transpose(2, 3)[..., None]).flatten(1, 2)

    k, v = gathered(s["k_cache"], s["k_scale"]), gathered(s["v_cache"], s["v_scale"])
    row = (starts[:-1, None] + torch.arange(width, device=dev)).clamp(max=q.shape[0] - 1)
    qs = q[row].float().unflatten(2, (-1, group))                       # [B, N, H, G, D]
    qs = qs.permute(0, 2, 1, 3, 4).flatten(2, 3)                        # [B, H, N G, D]
    scores = qs @ k.permute(0, 2, 3, 1) * dim ** -0.5                   # [B, H, N G, L]
    key = torch.arange(keys, device=dev)[None, :]
    draft = key - ctx[:, None]
    bit = (s["mask"][row, 0][:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
    seen = (draft < 0)[:, None, :] | ((draft >= 0) & (draft < new[:, None]))[:, None, :] & (bit == 1)
    seen = seen[:, None, :, None, :]
    scores = torch.where(seen, scores.unflatten(2, (width, group)), -math.inf)
    most = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - most)
    mass = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (width, group)) / mass
    lse = (most + torch.log(mass))[..., 0]
    b, i = s["request"], s["local"]
    return out[b, :, i].flatten(1, 2).to(q.dtype), lse[b, :, i].flatten(1, 2)


def _plain_sample(s):
    logits = s["logits"].double()
    rows, vocab = logits.shape
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    # likely tokens first, of equal ones the lowest index
    ordered, index = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.exp((ordered - ordered[:, :1]) / t)
    rank = torch.arange(vocab, device=logits.device)[None, :]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        w = torch.where((rank < k) | (k <= 0), w, 0.0)
    if s["min_p"] is not None:
        w = torch.where(w >= s["min_p"].double()[:, None], w, 0.0)
    if s["top_p"] is not None:
        top_p = s["top_p"].double()[:, None]
        before = torch.cumsum(w, 1) - w
        w = torch.where((before < top_p * w.sum(1, keepdim=True)) | (top_p >= 1), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, index, w)                            # in the order of the indices again
    mass = torch.cumsum(w, 1)
    token = (mass <= s["u"].double()[:, None] * mass[:, -1:]).sum(1)
    return torch.where(greedy, index[:, 0], token).to(torch.int32)


def _plain_accept(s):
    starts, width = s["row_start"].long(), s["max_new"]
    new = (starts[1:] - starts[:-1])[:, None]
    dev = starts.device
    at = torch.arange(width, device=dev)
    row = (starts[:-1, None] + at).clamp(max=s["tokens"].shape[0] - 1)
    tokens, target, parent = s["tokens"][row], s["target"][row], s["parents"][row].long()
    parent = parent.clamp(min=0)
    fits = (tokens == target.gather(1, parent)) & (at < new) & (at > 0)
    # of the drafts behind one token that fit, the first
    same = (parent[:, :, None] == parent[:, None, :]) & fits[:, None, :] & (at[None, :] < at[:, None])
    kept = (fits & ~same.any(2)) | (at == 0) & (new > 0)
    above = parent.masked_fill(at == 0, 0)
    for _ in range(max(1, (width - 1).bit_length())):                       # all ancestors, twice as many a step
        kept = kept & kept.gather(1, above)
        above = above.gather(1, above)
    order = torch.where(kept, at, width).sort(1)[0]
    length = kept.sum(1)
    path = torch.where(order < width, order, -1)
    last = path.gather(1, (length - 1).clamp(min=0)[:, None]).clamp(min=0)
    return path.to(torch.int32), length.to(torch.int32), target.gather(1, last)[:, 0]


def _kept(s):
    """What a user's program makes once and keeps: the handles of the cache and the rotation, and the workspace."""
    if "handles" not in s:
        from ternary_weight_linear_block_gb300 import binding, kv, sampling
        cache = rotary = None
        if "k_cache" in s:
            cache = (kv.KVCache8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]) if "k_scale" in s
                     else kv.KVCache(s["k_cache"], s["v_cache"]))
        if "freq" in s:
            rotary = kv.Rotary(s["freq"], axis=s["axis"] if s["case"]["axes"] > 1 else None,
                               neighbours=s["case"]["neighbours"])
        s["handles"] = kv, sampling, cache, rotary, binding.Workspace()
    return s["handles"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"rotate": _plain_rotate, "store": _plain_store, "attn": _plain_attn, "sample": _plain_sample,
                "accept": _plain_accept}[op](s)
    kv, sampling, cache, rotary, ws = _kept(s)
    if op == "sample":
        return sampling.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])
    if op == "accept":
        return sampling.accept(s["tokens"], s["target"], s["parents"], s["row_start"], s["max_new"])
    if op == "attn":
        return kv.tree_attention(s["q"], cache, s["table"], s["ctx_len"], s["row_start"], s["max_new"],
                                 mask=s["mask"], ws=ws, return_lse=True)
    if op == "store":
        kv.kv_write(cache, s["k"], s["v"], s["slots"])
        return kv.kv_read(cache, s["slots"], dtype=s["k"].dtype)
    q = kv.rotate_write(cache, s["q"], s["k"], s["v"], s["slots"], rotary, s["positions"], q_norm=s["q_norm"],
                        k_norm=s["k_norm"], eps=EPS)
    if s["case"]["cache"] in CODES:
        return (q,) + tuple(kv.kv_read(cache, s["slots"], dtype=s["k"].dtype))
    return q, s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "sample":
        cell = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * cell + 24), "flops": 0}
    ctx, new = _lengths(case)
    total = sum(new)
    if op == "accept":
        return {"bytes": 16 * total + 12 * case["requests"], "flops": 0}
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    row = heads * dim
    if op in ("store", "rotate"):
        # keys and values read once and written once; in 8 bits also their scales, and read back
        stored = 2 * total * (row + 4 * heads) if case["cache"] in CODES else 4 * total * row
        read = stored + 4 * total * row if case["cache"] in CODES else 0
        q = 4 * total * row * case["group"] if op == "rotate" else 0
        return {"bytes": 4 * total * row + stored + read + q + 8 * total, "flops": 0}
    q_heads = heads * case["group"]
    keys = sum(c + n for c, n in zip(ctx, new))
    pairs = sum((c + n) * n for c, n in zip(ctx, new))
    table = 4 * sum(_pages(c + n, page) for c, n in zip(ctx, new))
    return {"bytes": 2 * keys * (row + 4 * heads) + 4 * total * q_heads * dim + 12 * total * q_heads + table,
            "flops": 4 * pairs * q_heads * dim}


# ------------------------------------------------------------------ the definition, in 64 bits

def _stored(x, kind):
    """What rows of 64-bit values are as read from an 8-bit cache."""
    most = x.abs().amax(-1, keepdim=True)
    unit = most / LARGEST[kind]
    y = x / torch.where(unit > 0, unit, 1.0)
    step = torch.ones_like(y)
    if kind == "e4m3":                                            # 3 bits behind the first, down to 2^-9
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(most >= SMALLEST, torch.round(y / step) * step * unit, 0.0)


def exact(case, seed):
    op = case["op"]
    if op in ("sample", "accept"):
        return None                                                          # whole numbers alone
    s = prepare(case, seed)
    if op == "store":
        return _stored(s["k"].double(), case["cache"]), _stored(s["v"].double(), case["cache"])
    if op == "rotate":
        total, dim, rot, half = s["total"], case["dim"], case["rot"], case["rot"] // 2
        turn = torch.zeros(total, half, dtype=torch.complex128, device="cuda")
        for j in range(half):
            at = s["positions"][int(s["axis"][j])] if case["axes"] > 1 else s["positions"]
            angle = at.double() * float(s["freq"][j])
            turn[:, j] = torch.complex(torch.cos(angle), torch.sin(angle))
        pairs = [(2 * j, 2 * j + 1) if case["neighbours"] else (j, j + half) for j in range(half)]
        real, imag = [list(p) for p in zip(*pairs)]

        def turned(x, weight):
            x = x.double()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + EPS) * weight.double()
            z = torch.complex(x[..., real], x[..., imag]) * turn[:, None]
            y = x.clone()
            y[..., real], y[..., imag] = z.real, z.imag
            return y

        q, k, v = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"]), s["v"].double()
        if case["cache"] in CODES:
            return q, _stored(k, case["cache"]), _stored(v, case["cache"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.flatten(0, 1)[s["slots"]], vc.flatten(0, 1)[s["slots"]] = k, v
        return q, kc, vc
    ctx, new = _lengths(case)
    heads, group, dim, page = case["kv_heads"], case["group"], case["dim"], case["page"]
    out = torch.empty(s["total"], heads, group, dim, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["total"], heads, group, dtype=torch.float64, device="cuda")
    q = s["q"].unflatten(1, (heads, group))
    kc, vc = s["k_cache"].view(torch.int8), s["v_cache"].view(torch.int8)
    kind = CODES[case["cache"]]
    first = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        used = s["table"][b, :_pages(c + n, page)].long()
        hidden = torch.zeros(n, 1, c + n, dtype=torch.bool, device="cuda")
        for i, (word,) in enumerate(s["mask"][first:first + n].tolist()):
            hidden[i, 0, c:] = torch.tensor([not (word >> j) & 1 for j in range(n)], device="cuda")
        for h in range(heads):
            k = kc[used, :, h].view(kind).double() * s["k_scale"][used, h].double()[..., None]
            v = vc[used, :, h].view(kind).double() * s["v_scale"][used, h].double()[..., None]
            k, v = k.reshape(-1, dim)[:c + n], v.reshape(-1, dim)[:c + n]
            scores = torch.tensordot(q[first:first + n, h].double(), k, ([2], [1])) / math.sqrt(dim)
            scores.masked_fill_(hidden, -math.inf)
            lse[first:first + n, h] = torch.logsumexp(scores, -1)
            out[first:first + n, h] = torch.tensordot(torch.softmax(scores, -1), v, ([2], [0]))
        first += n
    return out.flatten(1, 2), lse.flatten(1, 2)
