"""The operators of a speculative step over a tree of drafted tokens, as cases that can be timed and checked.

Every case is one call that a serving program makes:

  rope      the step's queries and keys turned to their positions (one axis for text, three for images and video), the
            keys and values put into their slots of the paged cache
  tree      attention of the drafted tokens of each sequence over its paged cache: a token sees the context before the
            tree and its own ancestors
  verify    the path of drafted tokens that stands: a token drawn from the target's probabilities at each node, as long
            as it is one of that node's drafted children
  path      keys and values of the tokens that stand, moved to the positions that follow the context

``run`` computes a case with elementary torch operations in 32 bits or more; with ``own`` set it makes the framework's
calls instead.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
KSCALE, VSCALE = 1.0 / 64, 1.0 / 32   # what one unit of a code stands for in a quantised cache
CHILD = 0.7                           # probability that a drawn token is one of a node's drafted children
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 100 sequences: latency
        {"name": "rope_step_bf16", "op": "rope", "cache": "bf16", "tokens": 100, "heads": 64, "kv_heads": 8, "dim": 128,
         "rope_dim": 128, "axes": 1, "interleaved": False, "first": 8192, "block": 16},
        # a step's chunk of a long prompt into a quantised cache
        {"name": "rope_chunk_fp8", "op": "rope", "cache": "fp8", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rope_dim": 128, "axes": 1, "interleaved": False, "first": 100000, "block": 16},
        # the frames of a video: time, height and width, a rotary part of half the head
        {"name": "rope_video_f16", "op": "rope", "cache": "f16", "tokens": 5003, "heads": 32, "kv_heads": 32, "dim": 128,
         "rope_dim": 64, "axes": 3, "interleaved": True, "first": 0, "block": 32},
        # one chat request with a few drafts: latency
        {"name": "tree_one_bf16", "op": "tree", "cache": "bf16", "seqs": 1, "lo": 600, "hi": 600, "nodes": 8,
         "heads": 64, "kv_heads": 8, "dim": 128, "block": 16},
        # a full decode batch, sixteen drafted tokens a sequence
        {"name": "tree_batch_bf16", "op": "tree", "cache": "bf16", "seqs": 100, "lo": 8192, "hi": 8192, "nodes": 16,
         "heads": 64, "kv_heads": 8, "dim": 128, "block": 16},
        # contexts from a question to a book chapter over a quantised cache
        {"name": "tree_mix_fp8", "op": "tree", "cache": "fp8", "seqs": 64, "lo": 512, "hi": 16384, "nodes": 25,
         "heads": 32, "kv_heads": 8, "dim": 128, "block": 16},
        # a few long documents with wide trees
        {"name": "tree_wide_f16", "op": "tree", "cache": "f16", "seqs": 4, "lo": 32768, "hi": 32768, "nodes": 64,
         "heads": 64, "kv_heads": 8, "dim": 128, "block": 32},
        # a few interactive requests, small odd vocabulary
        {"name": "verify_few_f32", "op": "verify", "probs": "f32", "seqs": 4, "nodes": 16, "branch": 3, "vocab": 32003},
        # a full batch, large vocabulary
        {"name": "verify_batch_bf16", "op": "verify", "probs": "bf16", "seqs": 64, "nodes": 32, "branch": 2,
         "vocab": 131072},
        # one layer of a small batch: latency
        {"name": "path_few_bf16", "op": "path", "cache": "bf16", "seqs": 8, "nodes": 16, "layers": 1, "kv_heads": 8,
         "dim": 128, "block": 16},
        # every layer of a batch at once
        {"name": "path_layers_fp8", "op": "path", "cache": "fp8", "seqs": 64, "nodes": 32, "layers": 32, "kv_heads": 8,
         "dim": 128, "block": 16},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "verify", "path"])
    cache = rng.choice(["f16", "bf16", "fp8"])
    block = rng.choice([8, 16, 32])
    if op == "rope":
        heads, kv_heads = rng.choice([(64, 8), (32, 8), (32, 32), (16, 16), (5, 1), (12, 4)])
        dim = rng.choice([64, 80, 96, 128, 128])
        return {"op": op, "cache": cache, "tokens": _log(rng, 1, 8192), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rope_dim": rng.choice([dim, dim, 32, 64]), "axes": rng.choice([1, 1, 2, 3]),
                "interleaved": rng.choice([False, True]), "first": rng.choice([0, 1000, 131072, 1000000]),
                "block": block}
    if op == "tree":
        heads, kv_heads = rng.choice([(64, 8), (32, 8), (32, 32), (40, 8), (16, 1), (12, 4)])
        nodes = _log(rng, 1, 64)
        lo = _log(rng, nodes, 8192)
        hi = _log(rng, lo, 16384)
        most = max(1, min(64, 100000 // hi * (8 if kv_heads <= 8 else 2) // 8))
        return {"op": op, "cache": cache, "seqs": _log(rng, 1, most), "lo": lo, "hi": hi, "nodes": nodes,
                "heads": heads, "kv_heads": kv_heads, "dim": 128 if cache == "fp8" else rng.choice([64, 128, 128]),
                "block": block}
    if op == "verify":
        return {"op": op, "probs": rng.choice(["f32", "bf16", "f16"]), "seqs": _log(rng, 1, 48),
                "nodes": _log(rng, 1, 32), "branch": rng.choice([1, 2, 3, 4]), "vocab": _log(rng, 500, 131072) // 2}
    return {"op": op, "cache": cache, "seqs": _log(rng, 1, 64), "nodes": _log(rng, 4, 64),
            "layers": rng.choice([1, 2, 5, 16]), "kv_heads": rng.choice([1, 4, 8]), "dim": rng.choice([64, 128]),
            "block": block}


def _lens(case):
    """Contexts with their drafted tokens, spread evenly over their logarithm in a fixed shuffled order."""
    lo, hi = case["lo"], case["hi"]
    return [int(round(lo * (hi / lo) ** ((0.5 + i * 0.6180339887498949) % 1.0))) for i in range(case["seqs"])]


def _nodes(case):
    """Nodes of each sequence's tree; some requests bring fewer."""
    n = case["nodes"]
    return [n if i % 5 != 4 else n - n // 3 for i in range(case["seqs"])]


def _trees(case):
    """Each sequence's tree, parents before children: node 0 is the last known token, every node gets the same number
    of drafted children in turn (a chain with one), another number for each sequence."""
    return [[-1] + [(j - 1) // (1 + (i + case.get("branch", 2) - 1) % 4) for j in range(1, n)]
            for i, n in enumerate(_nodes(case))]


def _depth(tree):
    """Levels below a tree's root."""
    level = []
    for p in tree:
        level.append(0 if p < 0 else level[p] + 1)
    return max(level)


def _kept(case):
    """Drafted tokens that stand, of each sequence."""
    return [(3 + 2 * i) % (1 + min(8, (n - 1) // 2)) for i, n in enumerate(_nodes(case))]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def _cache(case, g, *shape):
    """A cache whose every slot holds a row."""
    x = _randn(g, *shape)
    if case["cache"] == "fp8":
        return (x * 64.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(DTYPES[case["cache"]])


def _held(cache):
    """What a cache holds: codes as the values that they are."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _tables(case, g, lens):
    """Number of blocks, and block tables of sequences placed over them at random."""
    need = [-(-n // case["block"]) for n in lens]
    nb = sum(need) + 3
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = ids[at:at + n]
        at += n
    return nb, tables


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    host = random.Random(int(seed) * 104729 + 7)
    s = {"case": case}
    if op == "rope":
        n, hq, hk, d, bs = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["block"]
        dt = DTYPES.get(case["cache"], torch.float16)
        # queries, keys and values as slices of one projection's rows; every 16th token is padding
        rows = _randn(g, n, hq + 2 * hk, d).to(dt)
        s["query"], s["key"], s["value"] = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
        nb = -(-n // bs) + 5
        slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n]
        slots[7::16] = -1
        s["slots"] = slots
        t = torch.arange(n, device=DEV) + case["first"] + host.randrange(100)
        if case["axes"] == 1:
            s["positions"] = t.to(torch.int32).view(1, n)
        else:   # frames of 20 x 25 patches
            s["positions"] = torch.stack([t // 500, t // 25 % 20, t % 25][:case["axes"]]).to(torch.int32)
        pairs = case["rope_dim"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)).float()
        s["pair_axis"] = (torch.arange(pairs, device=DEV) % case["axes"]).to(torch.int32)
        width = torch.uint8 if case["cache"] == "fp8" else dt
        s["k_cache"] = torch.zeros(nb, hk, bs, d, dtype=width, device=DEV)
        s["v_cache"] = torch.zeros(nb, hk, bs, d, dtype=width, device=DEV)
        s["out"] = torch.zeros(n, hq, d, dtype=dt, device=DEV)
    elif op == "tree":
        lens, trees = _lens(case), _trees(case)
        dt = DTYPES.get(case["cache"], torch.float16)
        nb, s["tables"] = _tables(case, g, lens)
        shape = (nb, case["kv_heads"], case["block"], case["dim"])
        s["k_cache"], s["v_cache"] = _cache(case, g, *shape), _cache(case, g, *shape)
        counts = [len(t) for t in trees]
        s["lens"], s["max_len"], s["start"] = _i32(lens), max(lens), _i32(_starts(counts))
        s["parents"] = _i32([p for t in trees for p in t])
        s["depth"], s["most"] = max(_depth(t) for t in trees), max(counts)
        s["query"] = _randn(g, sum(counts), case["heads"], case["dim"]).to(dt)
        s["scale"] = 1.0 / math.sqrt(case["dim"])
        s["out"] = torch.empty_like(s["query"])
    elif op == "verify":
        trees, v = _trees(case), case["vocab"]
        counts = [len(t) for t in trees]
        start, n, nb = _starts(counts), sum(counts), case["seqs"]
        dt = {"f32": torch.float32, **DTYPES}[case["probs"]]
        # a node's drafted children are likely tokens: together they have probability CHILD
        logits = 2.0 * _randn(g, n, v)
        tokens = [host.randrange(v) for _ in range(n)]
        at, col, up = [], [], []
        for i, t in enumerate(trees):
            kids = {}
            for j, p in enumerate(t):
                if p >= 0:
                    kids.setdefault(p, []).append(j)
            for p, js in kids.items():
                for j, token in zip(js, host.sample(range(v), len(js))):
                    tokens[start[i] + j] = token
                    at.append(start[i] + p)
                    col.append(token)
                    up.append(math.log(CHILD / (1 - CHILD) / len(js)))
        if at:
            rows = torch.tensor(at, device=DEV)
            rest = torch.logsumexp(logits, dim=1)
            logits[rows, torch.tensor(col, device=DEV)] = rest[rows] + torch.tensor(up, dtype=torch.float32, device=DEV)
        s["target"] = torch.softmax(logits, dim=1).to(dt)
        s["tokens_in"], s["parents"] = _i32(tokens), _i32([p for t in trees for p in t])
        s["start"], s["most"] = _i32(start), max(counts)
        s["depth"] = max(_depth(t) for t in trees)
        s["uniform"] = torch.rand(n, generator=g, device=DEV, dtype=torch.float32)
        s["accepted"] = torch.empty(nb, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(nb, s["depth"] + 1, dtype=torch.int32, device=DEV)
        s["path"] = torch.empty(nb, s["depth"] + 1, dtype=torch.int32, device=DEV)
    else:
        counts, kept = _nodes(case), _kept(case)
        lens = [n + 37 * i % 100 for i, n in enumerate(counts)]
        nb, s["tables"] = _tables(case, g, lens)
        shape = (case["layers"], nb, case["kv_heads"], case["block"], case["dim"])
        s["k_cache"], s["v_cache"] = _cache(case, g, *shape), _cache(case, g, *shape)
        s["lens"], s["start"] = _i32(lens), _i32(_starts(counts))
        # the nodes that stand, in order; beyond the first positions, so that a second pass finds them as they were
        paths = [[0] + sorted(host.sample(range(k + 1, n), k)) for n, k in zip(counts, kept)]
        s["path"] = _i32([p + [-1] * (max(kept) + 1 - len(p)) for p in paths])
        s["accepted"] = _i32(kept)
    return s


# ------------------------------------------------------------------ plain forms and the framework's calls

def _turn(x, cos, sin, interleaved):
    """Rows [n, heads, dim] as floats with their rotary part turned; cos and sin [n, pairs]."""
    x, pairs = x.float(), cos.shape[1]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    part, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = part[..., :pairs], part[..., pairs:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([part, rest], dim=-1)


def _rope(s):
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    bs = k_cache.shape[2]
    angle = s["positions"].double()[s["pair_axis"].long()].T * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    turned = s["case"]["interleaved"]
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    key = _turn(s["key"], cos, sin, turned)[keep]
    value = s["value"][keep].float()
    if k_cache.dtype == torch.uint8:
        key = (key / KSCALE).clamp(-448.0, 448.0)
        value = (value / VSCALE).clamp(-448.0, 448.0)
    _held(k_cache)[at // bs, :, at % bs] = key.to(_held(k_cache).dtype)
    _held(v_cache)[at // bs, :, at % bs] = value.to(_held(v_cache).dtype)
    query = _turn(s["query"], cos, sin, turned).to(s["out"].dtype)
    s["out"].copy_(torch.where(keep.view(-1, 1, 1), query, s["out"]))
    return [s["out"], _held(k_cache), _held(v_cache)]


def _tree(s):
    b, bs, dim = s["lens"].shape[0], s["k_cache"].shape[2], s["k_cache"].shape[3]
    nq, hq, _ = s["query"].shape
    hk, most = s["k_cache"].shape[1], s["most"]
    start, lens = s["start"].long(), s["lens"].long().view(b, 1)
    j = torch.arange(most, device=DEV)
    count = (start[1:] - start[:-1]).view(b, 1)
    row = torch.where(j < count, start[:-1].view(b, 1) + j, 0)
    # the nodes that each node sees: itself and its ancestors
    parents = s["parents"].long()[row]
    sees = torch.zeros(b, most, most + 1, dtype=torch.bool, device=DEV)
    node = j.repeat(b, 1)
    for _ in range(s["depth"] + 1):
        sees.scatter_(2, torch.where(node < 0, most, node).unsqueeze(2), True)
        node = torch.where(node < 0, -1, torch.gather(parents, 1, node.clamp(min=0)))
    # keys and values of every position
    pos = torch.arange(s["max_len"], device=DEV)
    blk = torch.where(pos < lens, s["tables"].long()[:, pos // bs], 0)
    k = _held(s["k_cache"])[blk, :, pos % bs].float().transpose(1, 2)       # [b, hk, positions, dim]
    v = _held(s["v_cache"])[blk, :, pos % bs].float().transpose(1, 2)
    scale = s["scale"]
    if s["k_cache"].dtype == torch.uint8:
        scale, v = scale * KSCALE, v * VSCALE
    g = hq // hk
    q = s["query"][row].float().view(b, most, hk, g, dim).permute(0, 2, 1, 3, 4).reshape(b, hk, most * g, dim)
    score = (torch.matmul(q, k.transpose(2, 3)) * scale).view(b, hk, most, g, -1)
    rel = pos - (lens - count)                                              # the node at each position
    in_tree = torch.gather(sees, 2, rel.clamp(0, most - 1).view(b, 1, -1).expand(b, most, -1))
    seen = (rel < 0).unsqueeze(1) | (in_tree & (rel < count).unsqueeze(1))  # [b, nodes, positions]
    score = score.masked_fill(~seen.view(b, 1, most, 1, -1), -math.inf)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    p = (p / p.sum(dim=-1, keepdim=True)).view(b, hk, most * g, -1)
    out = torch.matmul(p, v).view(b, hk, most, g, dim).permute(0, 2, 1, 3, 4).reshape(b, most, hq, dim)
    at = torch.arange(nq, device=DEV)
    seq = torch.searchsorted(start, at, right=True) - 1
    return out[seq, at - start[seq]].to(s["query"].dtype)


def _verify(s):
    nb, width = s["tokens"].shape
    start = s["start"].long()
    count = (start[1:] - start[:-1]).view(nb, 1)
    j = torch.arange(s["most"], device=DEV)
    row = torch.where(j < count, start[:-1].view(nb, 1) + j, 0)
    parents = torch.where(j < count, s["parents"].long()[row], -2)
    drafted = s["tokens_in"].long()[row]
    node = torch.zeros(nb, dtype=torch.long, device=DEV)
    going = torch.ones(nb, dtype=torch.bool, device=DEV)
    kept = torch.zeros(nb, dtype=torch.int32, device=DEV)
    tokens, path = [], []
    for level in range(width):
        at = start[:-1] + node
        c = s["target"][at].double().cumsum(dim=1)
        v = torch.searchsorted(c, s["uniform"].double()[at].view(nb, 1) * c[:, -1:], right=True)
        v = v.clamp(max=c.shape[1] - 1)
        tokens.append(torch.where(going, v.view(nb), -1))
        path.append(torch.where(going, node, -1))
        child = (parents == node.view(nb, 1)) & (drafted == v)
        going = going & child.any(dim=1) & (level + 1 < width)
        node = torch.where(going, child.long().argmax(dim=1), node)
        kept += going.int()
    return [kept, torch.stack(tokens, 1).to(torch.int32), torch.stack(path, 1).to(torch.int32)]


def _path(s):
    bs = s["k_cache"].shape[3]
    path, first = s["path"].long(), (s["lens"] - s["start"][1:] + s["start"][:-1]).long().view(-1, 1)
    j = torch.arange(path.shape[1], device=DEV)
    stands = j <= s["accepted"].view(-1, 1)
    src, dst = first + torch.where(stands, path, 0), first + torch.where(stands, j, 0)
    tables = s["tables"].long()
    sb, db = torch.gather(tables, 1, src // bs), torch.gather(tables, 1, dst // bs)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, db, :, dst % bs] = cache[:, sb, :, src % bs]
    return [_held(s["k_cache"]), _held(s["v_cache"])]


def _run_own(s):
    import paged_kv_cache_12_gb300 as pa

    case = s["case"]
    op = case["op"]
    scales = {"k_scale": KSCALE, "v_scale": VSCALE} if case.get("cache") == "fp8" else {}
    if op == "rope":
        pa.pa_kv_write_rope(s["key"], s["value"], s["positions"], s["inv_freq"], s["slots"], s["k_cache"], s["v_cache"],
                            query=s["query"], query_out=s["out"], pair_axis=s["pair_axis"],
                            interleaved=case["interleaved"], **scales)
        return [s["out"], _held(s["k_cache"]), _held(s["v_cache"])]
    if op == "tree":
        if "workspace" not in s:
            nq, hq, d = s["query"].shape
            size = pa.pa_attention_tree_workspace_size(s["lens"].shape[0], nq, hq, s["k_cache"].shape[1], d,
                                                       s["max_len"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        pa.pa_attention_tree(s["out"], s["query"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["start"],
                             s["parents"], s["scale"], s["max_len"], s["workspace"], **scales)
        return s["out"]
    if op == "verify":
        pa.pa_verify_tree(s["accepted"], s["tokens"], s["path"], s["target"], s["tokens_in"], s["parents"], s["start"],
                          s["uniform"])
        return [s["accepted"], s["tokens"], s["path"]]
    pa.pa_kv_move_path(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["start"], s["path"], s["accepted"])
    return [_held(s["k_cache"]), _held(s["v_cache"])]


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope, "tree": _tree, "verify": _verify, "path": _path}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    size = 1 if case.get("cache") == "fp8" else 2
    if op == "rope":
        n, hq, hk, d = (case[x] for x in ("tokens", "heads", "kv_heads", "dim"))
        real = n - (n + 8) // 16      # tokens that are not padding
        # a turned pair takes four products and two sums
        return {"bytes": real * d * (4 * hq + 2 * hk * (2 + size)) + n * (8 + 4 * case["axes"]) + 4 * case["rope_dim"],
                "flops": 3 * real * (hq + hk) * case["rope_dim"]}
    if op == "tree":
        lens, counts = _lens(case), _nodes(case)
        seen = 0                      # positions seen, over all nodes
        for n, t in zip(lens, _trees(case)):
            level = []
            for p in t:
                level.append(1 if p < 0 else level[p] + 1)
            seen += len(t) * (n - len(t)) + sum(level)
        return {"bytes": sum(lens) * 2 * case["kv_heads"] * case["dim"] * size
                + sum(counts) * (4 * case["heads"] * case["dim"] + 4) + 4 * sum(-(-x // case["block"]) for x in lens),
                "flops": 4 * case["heads"] * case["dim"] * seen}
    if op == "verify":
        rows = 0.0                    # rows of the target that are looked at, on average
        for t in _trees(case):
            kids = [t.count(j) for j in range(len(t))]
            reach = []
            for p in t:
                reach.append(1.0 if p < 0 else reach[p] * CHILD / kids[p])
            rows += sum(reach)
        width = 4 if case["probs"] == "f32" else 2
        return {"bytes": int(rows * case["vocab"] * width) + 8 * sum(_nodes(case)), "flops": 0}
    moved = sum(_kept(case))
    return {"bytes": moved * case["layers"] * case["kv_heads"] * case["dim"] * size * 2 * 2 + 8 * case["seqs"],
            "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _value_of(code):
    """The value of E4M3 codes (bytes as whole numbers): sign, four exponent bits of bias 7, three mantissa bits."""
    sign = 1.0 - 2.0 * (code >> 7).double()
    e, m = ((code >> 3) & 15).double(), (code & 7).double()
    return sign * torch.where(e > 0, torch.exp2(e - 7.0) * (1.0 + m / 8.0), m * 2.0 ** -9)


def _values(cache):
    """What a cache's elements are, in 64 bits (codes in units of their scale)."""
    return _value_of(cache.long()) if cache.dtype == torch.uint8 else cache.double()


def _nearest_code_value(y):
    """The nearest E4M3 value to each y, at most 448, ties to the even mantissa."""
    y = y.clamp(-448.0, 448.0)
    e = torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -6)))
    step = torch.exp2(torch.clamp(e, max=8.0) - 3.0)
    return torch.round(y / step) * step


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        n, d, r, bs = case["tokens"], case["dim"], case["rope_dim"], case["block"]
        i = torch.arange(d, device=DEV)
        # the partner of each element, and which pair it belongs to
        if case["interleaved"]:
            pair, other, first = i // 2, i ^ 1, i % 2 == 0
        else:
            pair, other, first = i % (r // 2), (i + r // 2) % r, i < r // 2
        inside = i < r
        pair, other = torch.where(inside, pair, 0), torch.where(inside, other, i)
        axis = s["pair_axis"].long()[pair]
        angle = s["positions"].double()[axis].T * s["inv_freq"].double()[pair]           # [n, d]
        cos = torch.where(inside, torch.cos(angle), 1.0).view(n, 1, d)
        sin = torch.where(inside, torch.where(first, -1.0, 1.0) * torch.sin(angle), 0.0).view(n, 1, d)
        rotated = {x: s[x].double() * cos + s[x].double()[..., other] * sin for x in ("query", "key")}
        real = [t for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
        blk, off = s["slots"][real] // bs, s["slots"][real] % bs
        out = torch.zeros(n, case["heads"], d, dtype=torch.float64, device=DEV)
        out[real] = rotated["query"][real]
        got = [out]
        for rows, unit in ((rotated["key"], KSCALE), (s["value"].double(), VSCALE)):
            held = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=DEV)
            held[blk, :, off] = _nearest_code_value(rows[real] / unit) if case["cache"] == "fp8" else rows[real]
            got.append(held)
        return got
    if op == "tree":
        hq, hk, bs = case["heads"], case["kv_heads"], case["block"]
        got, start = [], s["start"].tolist()
        units = (KSCALE, VSCALE) if case["cache"] == "fp8" else (1.0, 1.0)
        for i, (n, t) in enumerate(zip(_lens(case), _trees(case))):
            hide = torch.zeros(len(t), n, dtype=torch.bool, device=DEV)
            for j in range(len(t)):
                line, a = [], j
                while a >= 0:
                    line.append(n - len(t) + a)
                    a = t[a]
                hide[j, n - len(t):] = True
                hide[j, line] = False
            pos = torch.arange(n, device=DEV)
            blk = s["tables"][i].long()[pos // bs]
            k, v = (_values(s[x][blk, :, pos % bs]) * u for x, u in zip(("k_cache", "v_cache"), units))
            q = s["query"][start[i]:start[i + 1]].double()
            heads = []
            for h in range(hq):
                score = (q[:, h] @ k[:, h * hk // hq].T * s["scale"]).masked_fill(hide, -math.inf)
                heads.append(torch.softmax(score, 1) @ v[:, h * hk // hq])
            got.append(torch.stack(heads, 1))
        return torch.cat(got)
    if op == "verify":
        width, start = s["depth"] + 1, s["start"].tolist()
        drafted, u = s["tokens_in"].tolist(), s["uniform"].double().tolist()
        kept = np.zeros(case["seqs"], dtype=np.int32)
        tokens, path = (np.full((case["seqs"], width), -1, dtype=np.int32) for _ in range(2))
        for i, t in enumerate(_trees(case)):
            node = 0
            while True:
                at = start[i] + node
                c = np.cumsum(s["target"][at].double().cpu().numpy())
                v = int(np.searchsorted(c, u[at] * c[-1], side="right"))
                tokens[i, kept[i]], path[i, kept[i]] = v, node
                kids = [j for j, p in enumerate(t) if p == node and drafted[start[i] + j] == v]
                if not kids or kept[i] + 1 == width:
                    break
                node = kids[0]
                kept[i] += 1
        return [kept, tokens, path]
    got, bs = [], case["block"]
    for cache in (s["k_cache"], s["v_cache"]):
        before, after = _values(cache), _values(cache)
        for i, (n, m, k) in enumerate(zip(s["lens"].tolist(), _nodes(case), _kept(case))):
            for j in range(k + 1):
                src, dst = n - m + int(s["path"][i, j]), n - m + j
                after[:, int(s["tables"][i, dst // bs]), :, dst % bs] = \
                    before[:, int(s["tables"][i, src // bs]), :, src % bs]
        got.append(after)
    return got
