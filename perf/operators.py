"""The paged key/value cache and the verification of drafted token trees: the cases that are measured.

Four operators, as one step of speculative decoding uses them between the qkv and the output linear:

* ``plan``: block tables, slot maps and row starts on the GPU from the requests' lengths;
* ``write``: the new tokens' keys and values into the cache's slots;
* ``attn``: attention of every request's tree of drafted tokens over its cached tokens and its tree;
* ``commit``: the accepted path of each tree made contiguous in the caches of all layers.

``run`` is the plain form (32-bit torch operations, rounded once) or, where ``own`` is true, the calls that a
user makes of the framework.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's plan: 16 requests, up to 16 drafted tokens each
        dict(name="plan decode", op="plan", requests=16, new=16, ctx=4000, page=16),
        # a long prompt pass over many requests: about a million new tokens
        dict(name="plan prompts", op="plan", requests=1024, new=1511, ctx=700, page=16),
        # the 16 tokens of one decode step of the 5120-wide model (20 key heads of 128)
        dict(name="write decode", op="write", requests=2, new=8, ctx=1000, page=16, kv_heads=20, group=2, dim=128,
             dtype="bf16"),
        # a prompt pass: 65521 tokens, 8 key heads
        dict(name="write prompts", op="write", requests=13, new=9001, ctx=77, page=64, kv_heads=8, group=4,
             dim=128, dtype="bf16"),
        # 16 requests of one token each at short contexts: the smallest call, latency counts
        dict(name="attn one token", op="attn", requests=16, new=1, ctx=700, page=16, kv_heads=20, group=2, dim=128,
             dtype="bf16"),
        # ordinary serving: 64 requests of one token at uneven contexts
        dict(name="attn batch", op="attn", requests=64, new=1, ctx=16001, page=16, kv_heads=8, group=4, dim=128,
             dtype="bf16"),
        # one long conversation, a tree of 16 drafts
        dict(name="attn long", op="attn", requests=1, new=16, ctx=131001, page=64, kv_heads=8, group=4, dim=128,
             dtype="bf16"),
        # wide trees and many query heads on each key head: the most arithmetic for each byte
        dict(name="attn wide tree", op="attn", requests=4, new=64, ctx=32768, page=32, kv_heads=8, group=8, dim=128,
             dtype="fp16"),
        # head size 256, few key heads, odd tree sizes
        dict(name="attn d256", op="attn", requests=8, new=29, ctx=20003, page=128, kv_heads=2, group=8, dim=256,
             dtype="bf16"),
        # head size 64, one query head on each key head
        dict(name="attn d64", op="attn", requests=16, new=23, ctx=4099, page=16, kv_heads=16, group=1, dim=64,
             dtype="fp16"),
        # the accepted paths of one decode step, 16 layers
        dict(name="commit decode", op="commit", requests=2, new=8, ctx=200, page=16, kv_heads=20, group=2, dim=128,
             dtype="bf16", layers=16),
        # many requests with wide trees, 16 layers
        dict(name="commit batch", op="commit", requests=61, new=64, ctx=150, page=32, kv_heads=8, group=4, dim=128,
             dtype="bf16", layers=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "commit", "attn", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        requests = _log(rng, 1, 1024)
        return dict(op=op, requests=requests, new=_log(rng, 1, min(16384, 1500000 // requests)),
                    ctx=_log(rng, 1, 8000), page=page)
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 20])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    case = dict(op=op, page=page, kv_heads=kv_heads, group=group, dim=dim, dtype=rng.choice(["bf16", "fp16"]))
    row = kv_heads * dim
    if op == "write":
        requests = _log(rng, 1, 64)
        return dict(case, requests=requests, new=_log(rng, 1, max(1, 60000000 // (row * requests))),
                    ctx=_log(rng, 1, 300))
    if op == "commit":
        requests = _log(rng, 1, 48)
        return dict(case, requests=requests, new=_log(rng, 2, max(2, min(64, 3000000 // (row * requests)))),
                    ctx=_log(rng, 1, 150), layers=rng.choice([1, 3, 8, 16]))
    requests = _log(rng, 1, 128)
    new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 64)])
    # at most the wide tree's keys and arithmetic
    most = min(1.3e8 / (requests * row), 6.0e10 / (requests * new * group * row), 131072)
    return dict(case, requests=requests, new=new, ctx=_log(rng, 1, max(1, most)))


def _lengths(case):
    """Cached and new tokens of every request: uneven, by the case alone, the largest as the case says."""
    rng = random.Random("%(op)s %(requests)d %(new)d %(ctx)d %(page)d" % case)
    ctx = [max(1, int(case["ctx"] * rng.uniform(0.25, 1.0))) for _ in range(case["requests"])]
    new = [max(1, int(math.ceil(case["new"] * rng.uniform(0.5, 1.0)))) for _ in range(case["requests"])]
    ctx[-1], new[-1] = case["ctx"], case["new"]
    return ctx, new


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ inputs

def _signed(word):
    return word - (1 << 64) if word >= 1 << 63 else word


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ctx, new = _lengths(case)
    page, requests = case["page"], case["requests"]
    total = sum(new)
    int32 = dict(dtype=torch.int32, device=dev)
    held = [_pages(c, page) for c in ctx]
    needed = [_pages(c + n, page) for c, n in zip(ctx, new)]
    width = max(needed) + 1
    count = sum(needed)
    pages = count + 8
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    s = dict(case=case, total=total, page=page, pages=pages, max_new=max(new),
             ctx_len=torch.tensor(ctx, **int32), new_len=torch.tensor(new, **int32))
    if case["op"] == "plan":
        taken = sum(held)
        at = torch.arange(width, device=dev)[None, :]
        first = torch.tensor([0] + held[:-1], device=dev).cumsum(0)[:, None]
        known = at < torch.tensor(held, device=dev)[:, None]
        s["table"] = torch.where(known, order[(first + at).clamp(max=pages - 1)], -1).to(torch.int32)
        s["free"] = order[taken:].contiguous()
        s["capacity"] = total
        return s
    at = torch.arange(width, device=dev)[None, :]
    first = torch.tensor([0] + needed[:-1], device=dev).cumsum(0)[:, None]
    known = at < torch.tensor(needed, device=dev)[:, None]
    s["table"] = torch.where(known, order[(first + at).clamp(max=pages - 1)], 0).to(torch.int32)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["row_start"] = torch.tensor(starts, **int32)
    dtype, heads, dim = TYPES[case["dtype"]], case["kv_heads"], case["dim"]
    layers = case.get("layers", 1)
    q_heads = heads * case["group"]

    def tree(n, key):
        """A drafted tree: parent of each token (-1: the context), and each token's ancestors as bits."""
        rng, bits = random.Random(key), []
        parent = [-1] + [rng.randrange(max(0, i - 6), i) for i in range(1, n)]
        for i, p in enumerate(parent):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        return parent, bits

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    # keys have a few channels of large mean, as trained models' keys have
    mean = torch.zeros(heads, dim, device=dev, dtype=dtype)
    mean[:, torch.randperm(dim, generator=gen, device=dev)[:4]] = 3.0
    s["k_cache"] = normal(layers * pages, page, heads, dim).add_(mean)
    s["v_cache"] = normal(layers * pages, page, heads, dim)
    request = torch.repeat_interleave(torch.arange(requests, device=dev), s["new_len"].long())
    s["local"] = torch.arange(total, device=dev) - s["row_start"].long()[request]
    s["request"] = request
    position = s["ctx_len"].long()[request] + s["local"]
    slots = s["table"][request, position // page].long() * page + position % page
    s["slots"] = torch.cat([slots + layer * pages * page for layer in range(layers)])
    # queries, keys and values as the qkv linear leaves them: slices of one row
    if case["op"] == "attn":
        qkv = normal(total, (q_heads + 2 * heads) * dim)
        s["q"] = qkv[:, :q_heads * dim].unflatten(1, (q_heads, dim))
        trees = [tree(n, seed * 1000003 + b) for b, n in enumerate(new)]
        s["mask"] = torch.tensor([[_signed(w)] for _, bits in trees for w in bits], dtype=torch.int64, device=dev)
        return s
    kv = normal(layers * total, 2 * heads * dim)
    s["k"] = kv[:, :heads * dim].unflatten(1, (heads, dim))
    s["v"] = kv[:, heads * dim:].unflatten(1, (heads, dim))
    if case["op"] == "commit":
        paths, counts = [], []
        for b, n in enumerate(new):
            parent, _ = tree(n, seed * 1000003 + b)
            leaf, path = random.Random(seed * 7919 + b).randrange(n), []
            while leaf >= 0:
                path.append(leaf)
                leaf = parent[leaf]
            paths.append(path[::-1] + [0] * (max(new) - len(path)))
            counts.append(len(path))
        s["path"], s["path_len"] = torch.tensor(paths, **int32), torch.tensor(counts, **int32)
    return s


# ------------------------------------------------------------------ one pass

def _plain_plan(s):
    page, table, free = s["page"], s["table"], s["free"]
    ctx, new = s["ctx_len"], s["new_len"]
    dev = table.device
    held, needed = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    more = needed - held
    before = torch.cumsum(more, 0) - more
    at = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (at >= held[:, None]) & (at < needed[:, None])
    index = torch.where(fresh, before[:, None] + at - held[:, None], 0)
    table.copy_(torch.where(fresh, free[index], table))
    starts = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), torch.cumsum(new, 0, dtype=torch.int32)])
    token = torch.arange(s["capacity"], device=dev)
    request = torch.searchsorted(starts[1:], token.int(), right=True)
    position = (ctx[request] + token - starts[request]).int()
    slots = table[request, position // page].long() * page + position % page
    return table, starts, slots, position, request.int()


def _plain_write(s):
    k, v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    k[s["slots"]] = s["k"]
    v[s["slots"]] = s["v"]
    return s["k_cache"], s["v_cache"]


def _plain_attn(s):
    case, table, q, page = s["case"], s["table"], s["q"], s["page"]
    dev, dim, group = q.device, case["dim"], case["group"]
    starts, ctx, width = s["row_start"].long(), s["ctx_len"].long(), s["max_new"]
    new = starts[1:] - starts[:-1]
    requests, keys = table.shape[0], table.shape[1] * page
    k = s["k_cache"][table.long()].flatten(1, 2).float()                # [B, L, H, D]
    v = s["v_cache"][table.long()].flatten(1, 2).float()
    row = (starts[:-1, None] + torch.arange(width, device=dev)).clamp(max=q.shape[0] - 1)
    qs = q[row].float().unflatten(2, (-1, group))                       # [B, N, H, G, D]
    qs = qs.permute(0, 2, 1, 3, 4).flatten(2, 3)                        # [B, H, N G, D]
    scores = qs @ k.permute(0, 2, 3, 1) * dim ** -0.5                   # [B, H, N G, L]
    key = torch.arange(keys, device=dev)[None, :]
    draft = key - ctx[:, None]
    bit = (s["mask"][row, 0][:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
    seen = (draft < 0)[:, None, :] | ((draft >= 0) & (draft < new[:, None]))[:, None, :] & (bit == 1)
    seen = seen[:, None, :, None, :]
    scores = scores.unflatten(2, (width, group))
    scores = torch.where(seen, scores, -math.inf)
    most = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - most)
    mass = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (width, group)) / mass
    lse = (most + torch.log(mass))[..., 0]
    b, i = s["request"], s["local"]
    return out[b, :, i].flatten(1, 2).to(q.dtype), lse[b, :, i].flatten(1, 2)


def _plain_commit(s):
    _plain_write(s)                                                      # the step's drafts, all layers
    page, pages, table, ctx = s["page"], s["pages"], s["table"].long(), s["ctx_len"].long()
    layers, width = s["case"]["layers"], s["path"].shape[1]
    at = torch.arange(width, device=table.device)[None, :]
    keep = at < s["path_len"][:, None]
    last = table.shape[1] * page - 1
    source, target = (ctx[:, None] + s["path"]).clamp(max=last), (ctx[:, None] + at).clamp(max=last)
    source = torch.gather(table, 1, source // page) * page + source % page
    target = torch.gather(table, 1, target // page) * page + target % page
    source = torch.where(keep, source, target)                            # past the path: nothing moves
    layer = torch.arange(layers, device=table.device)[:, None, None] * (pages * page)
    source, target = (layer + source).flatten(), (layer + target).flatten()
    k, v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    # the padding of a path may stand on another token's place, so only the path itself is written
    chosen = keep.expand(layers, -1, -1).flatten()[:, None, None]
    drop = torch.where(chosen[:, 0, 0], target, k.shape[0])
    k2 = torch.cat([k, k[:1]])
    v2 = torch.cat([v, v[:1]])
    k2[drop] = k[source]
    v2[drop] = v[source]
    k.copy_(k2[:-1])
    v.copy_(v2[:-1])
    return s["k_cache"], s["v_cache"], s["ctx_len"] + s["path_len"]


def _kept(s):
    """What a user's program makes once and keeps: the handles of the caches and the workspace."""
    if "handles" not in s:
        from ternary_weight_linear_block_gb300 import binding, kv
        whole = layers = None
        if "k_cache" in s:
            whole = kv.KVCache(s["k_cache"], s["v_cache"])
            layers = [kv.KVCache(k, v) for k, v in zip(s["k_cache"].split(s["pages"]), s["v_cache"].split(s["pages"]))]
        s["handles"] = kv, whole, layers, binding.Workspace()
    return s["handles"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "write": _plain_write, "attn": _plain_attn, "commit": _plain_commit}[op](s)
    kv, whole, layers, ws = _kept(s)
    if op == "plan":
        p = kv.kv_plan(s["ctx_len"], s["new_len"], s["table"], s["free"], s["page"], s["capacity"])
        return s["table"], p.row_start, p.slots, p.positions, p.request
    if op == "attn":
        return kv.tree_attention(s["q"], whole, s["table"], s["ctx_len"], s["row_start"], s["max_new"],
                                 mask=s["mask"], ws=ws, return_lse=True)
    kv.kv_write(whole, s["k"], s["v"], s["slots"])
    if op == "write":
        return s["k_cache"], s["v_cache"]
    ctx = kv.kv_commit(layers, s["table"], s["ctx_len"], s["path"], s["path_len"])
    return s["k_cache"], s["v_cache"], ctx


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    ctx, new = _lengths(case)
    page, total = case["page"], sum(new)
    table = 4 * sum(_pages(c + n, page) for c, n in zip(ctx, new))
    if case["op"] == "plan":
        return {"bytes": 12 * case["requests"] + 16 * total + table, "flops": 0}
    row = case["kv_heads"] * case["dim"] * 2
    if case["op"] == "write":
        return {"bytes": 4 * total * row + 8 * total, "flops": 0}
    if case["op"] == "commit":
        # each draft written, and about a third of a path's tokens moved
        depth = sum(max(1, n // 6) for n in new)
        return {"bytes": (4 * total * row + 4 * depth * row) * case["layers"], "flops": 0}
    q_heads = case["kv_heads"] * case["group"]
    keys = sum(c + n for c, n in zip(ctx, new))
    pairs = sum((c + n) * n for c, n in zip(ctx, new))
    return {"bytes": 2 * keys * row + 4 * total * q_heads * case["dim"] + 12 * total * q_heads + table,
            "flops": 4 * pairs * q_heads * case["dim"]}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    if case["op"] == "plan":
        return None                                                      # whole numbers alone
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    page, op = case["page"], case["op"]
    kc, vc, table = s["k_cache"], s["v_cache"], s["table"].tolist()
    if op in ("write", "commit"):
        layers, pages, total = case.get("layers", 1), s["pages"], s["total"]
        kc, vc = kc.double().flatten(0, 1), vc.double().flatten(0, 1)
        for layer in range(layers):
            first = 0
            for b, (c, n) in enumerate(zip(ctx, new)):
                place = [(layer * pages + table[b][(c + i) // page]) * page + (c + i) % page for i in range(n)]
                rows = slice(layer * total + first, layer * total + first + n)
                kc[place], vc[place] = s["k"][rows].double(), s["v"][rows].double()
                if op == "commit":
                    path = s["path"][b, :int(s["path_len"][b])].tolist()
                    kept = [place[i] for i in path]
                    kc[place[:len(path)]], vc[place[:len(path)]] = kc[kept], vc[kept]
                first += n
        shape = s["k_cache"].shape
        both = kc.view(shape), vc.view(shape)
        return both if op == "write" else both + (None,)
    out = torch.empty(s["total"], case["kv_heads"], case["group"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.empty(s["total"], case["kv_heads"], case["group"], dtype=torch.float64, device="cuda")
    q = s["q"].unflatten(1, (case["kv_heads"], case["group"]))
    first = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        used = s["table"][b, :_pages(c + n, page)].long()
        hidden = torch.zeros(n, 1, c + n, dtype=torch.bool, device="cuda")
        for i, (word,) in enumerate(s["mask"][first:first + n].tolist()):
            hidden[i, 0, c:] = torch.tensor([not (word >> j) & 1 for j in range(n)], device="cuda")
        for h in range(case["kv_heads"]):
            k = kc[used, :, h].reshape(-1, case["dim"])[:c + n].double()
            v = vc[used, :, h].reshape(-1, case["dim"])[:c + n].double()
            scores = torch.tensordot(q[first:first + n, h].double(), k, ([2], [1])) / math.sqrt(case["dim"])
            scores.masked_fill_(hidden, -math.inf)
            lse[first:first + n, h] = torch.logsumexp(scores, -1)
            out[first:first + n, h] = torch.tensordot(torch.softmax(scores, -1), v, ([2], [0]))
        first += n
    return out.flatten(1, 2), lse.flatten(1, 2)
