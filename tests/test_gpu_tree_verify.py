"""pa_verify_tree against the definition in 64 bits (counts, tokens and nodes have
to be equal: decisions lie far from their borders compared with the kernel's
rounding, twice a float's precision), pa_kv_move_path against a copy of rows, and a
whole step over trees."""
import math
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa
import tree_ref as TR

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def tree_case(kind, counts, vocab, seed, width=None, likely=0.75):
    """Trees whose nodes' children together are likely tokens."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    start, n = [0] + np.cumsum(counts).tolist(), sum(counts)
    p = torch.softmax(2 * torch.randn(n, vocab, generator=g, device=DEV), 1)
    parents, tokens = [], []
    for i, c in enumerate(counts):
        t = TR.random_tree(rng, c, TR.KINDS[i % 4]) if c else []
        tok = [int(x) for x in rng.integers(0, vocab, c)]
        for j in range(c):
            kids = [x for x in range(j + 1, c) if t[x] == j]
            if kids:
                pick = rng.choice(vocab, size=len(kids), replace=len(kids) > vocab)
                row = p[start[i] + j]
                row *= 1 - likely
                for x, v in zip(kids, pick):
                    tok[x] = int(v)
                    row[int(v)] += likely / len(kids)
        parents += t
        tokens += tok
    width = width or vocab
    target = torch.full((n, width), math.nan, dtype=TYPES[kind], device=DEV)
    target[:, :vocab] = p.to(TYPES[kind])
    return target[:, :vocab], tokens, parents, start, rng.random(n).astype(np.float32)


def run(target, tokens, parents, start, u, depth, stream=None):
    b = len(start) - 1
    acc = torch.full((b,), -9, dtype=torch.int32, device=DEV)
    tok, path = (torch.full((b, depth + 1), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    pa.pa_verify_tree(acc, tok, path, target, i32(tokens), i32(parents), i32(start),
                      torch.tensor(np.asarray(u), dtype=torch.float32, device=DEV), stream=stream)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), tok.cpu().numpy(), path.cpu().numpy()


def compare(args, depth):
    target, tokens, parents, start, u = args
    got = run(*args, depth)
    want = TR.verify_tree(target.double().cpu().numpy(), tokens, parents, start, np.asarray(u, dtype=np.float64), depth)
    for x, y in zip(got, want):
        assert x.tolist() == y.tolist()
    return got


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("vocab,width", [(1, 1), (2, 2), (5, 8), (127, 127), (128, 128), (129, 132), (1000, 1000),
                                         (32003, 32003), (65537, 65544), (131072, 131072)])
def test_against_the_definition(kind, vocab, width):
    counts = [5, 1, 16, 0, 8, 3, 20, 9]
    acc, _, _ = compare(tree_case(kind, counts, vocab, vocab + 1, width), 6)
    assert acc[3] == -1


@pytest.mark.parametrize("b", [1, 70, 80, 160, 320, 700])
def test_batches_of_every_cluster_size(b):
    rng = np.random.default_rng(b)
    acc, _, _ = compare(tree_case("f32", [int(x) for x in rng.integers(1, 6, b)], 700, b), 4)
    assert b < 70 or len(set(acc.tolist())) >= 3


@pytest.mark.parametrize("b", [2, 90, 200, 400])
def test_long_slices_of_every_cluster_size(b):
    compare(tree_case("bf16", [3] * b, 40011 if b < 100 else 9001, b + 1), 3)


def test_depths():
    args = tree_case("f32", [12] * 12, 50, 3, likely=0.97)
    deep = [compare(args, depth)[0].max() for depth in (0, 1, 2, 5, 11, 40)]
    assert deep[0] == 0 and deep[1] == 1 and deep[4] > 3 and deep[5] == deep[4]


def test_trees_of_many_nodes():
    # more nodes than are kept in shared memory, paths deeper than a wave
    acc, _, _ = compare(tree_case("f32", [700, 300, 257, 5], 60, 21, likely=0.95), 40)
    assert acc.max() > 8


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts,vocab", [([8], 600011), ([8, 7, 8], 280000), ([17, 16], 1100003)])
def test_slices_longer_than_a_search(kind, counts, vocab):
    # a CTA a node and so many tokens that the passing slice is cut before it is searched
    for seed in (5, 6):
        compare(tree_case(kind, counts, vocab, seed, width=vocab + 3), 6)


@pytest.mark.parametrize("order", ["depth first", "a node's children 700 behind it", "backward"])
def test_numberings_of_trees(order):
    # waves take descendants by their numbers: paths through trees whose numbers say little
    n = 900
    if order == "depth first":        # chains of 30 from the root
        parents = [-1] + [0 if j % 30 == 1 else j - 1 for j in range(1, n)]
    elif order == "backward":         # parents that come after their children are nobody's
        parents = [-1] + [j + 1 if j % 3 == 0 else j // 3 for j in range(1, n)]
    else:
        parents = [-1] + [0 if j <= 700 else j - 700 for j in range(1, n)]
    g = torch.Generator().manual_seed(4)
    target = torch.softmax(torch.randn(8 * n, 2, generator=g), 1).to(DEV)
    tokens = np.random.default_rng(4).integers(0, 2, 8 * n).tolist()
    u = np.random.default_rng(5).random(8 * n).astype(np.float32)
    acc, _, _ = compare((target, tokens, parents * 8, [i * n for i in range(9)], u), 40)
    assert acc.max() > 1


def test_siblings_of_one_token_and_foreign_nodes():
    # the first of two children with the same token stands; a node without a parent is nobody's child
    p = torch.zeros(5, 8, device=DEV)
    p[:, 3] = 1.0
    got = compare((p, [0, 3, 3, 3, 3], [-1, -1, 0, 0, 2], [0, 5], [0.5] * 5), 4)
    assert got[2].tolist() == [[0, 2, 4, -1, -1]] and got[1].tolist() == [[3, 3, 3, -1, -1]]
    # parents out of range and drafted tokens outside the vocabulary match nothing
    got = compare((p, [0, -1, 8, 3, 3], [-1, 0, 0, 77, -9], [0, 5], [0.5] * 5), 4)
    assert got[0].tolist() == [0]


def test_rows_without_weight():
    p = torch.rand(6, 40, device=DEV)
    p[0] = 0
    p[1, 5], p[2, 7], p[3] = math.nan, -1.0, math.nan
    p[4, 3] = math.inf
    start = list(range(7))
    got = compare((p, [0] * 6, [-1] * 6, start, [0.1, 0.2, 0.3, 0.4, 0.5, 0.0]), 2)
    assert got[1][:, 0].tolist()[0] == -1 and got[1][3, 0] == -1 and got[1][4, 0] == -1


@pytest.mark.parametrize("kind,low", [("f32", -120), ("f16", -24), ("bf16", -120)])
@pytest.mark.parametrize("seqs,vocab", [(700, 40003), (2, 300007), (20, 20004)])
def test_weights_of_many_sizes(kind, low, seqs, vocab):
    # rising rows (each step's largest passes the sum before it), falling and mixed ones,
    # with negative elements, NaN and one infinity among them.  Powers of two: the 64-bit
    # sums here are exact to 2^-53 of the total, the kernel's to about 2^-44, and a
    # number of 24 bits falls within 2^-40 of one of the few sums above 2^-24 of the total
    # with a probability below 1e-5.
    rng = np.random.default_rng(seqs)
    x = np.sort(np.exp2(rng.integers(low, 1, (seqs, vocab)).astype(np.float64)), axis=1)
    x[1::3] = x[1::3, ::-1]
    for i in range(2, seqs, 3):
        rng.shuffle(x[i])
    for i in range(0, seqs, 4):
        at = rng.integers(0, vocab, 9)
        x[i, at[:4]], x[i, at[4:8]] = math.nan, -0.5
        if i % 8:
            x[i, at[8]] = math.inf
    target = torch.from_numpy(x).to(TYPES[kind]).to(DEV)
    u = rng.random(seqs).astype(np.float32)
    got = compare((target, [0] * seqs, [-1] * seqs, list(range(seqs + 1)), u), 0)
    assert all((got[1][i, 0] == -1) == (i % 8 == 4) for i in range(seqs))


def test_bad_tree_start():
    target, tokens, parents, _, u = tree_case("f32", [4, 4, 4], 30, 2)
    for start in ([0, 5, 4, 12], [1, 4, 8, 12], [0, 4, 8, 11], [0, 4, 8, 13], [0, -4, 8, 12]):
        acc, tok, path = run(target, tokens, parents, start, u, 3)
        n = 12
        for i in range(3):
            a, b = start[i], start[i + 1]
            ok = 0 <= a < b <= n and (i > 0 or a == 0) and (i < 2 or b == n)
            if not ok:
                assert acc[i] == -1 and (tok[i] == -1).all() and (path[i] == -1).all()


def test_chain_agrees_with_pa_verify_drafts_without_draft_rows():
    # a chain of one draft: the draft stands exactly when the drawn token is the draft
    target, tokens, parents, start, u = tree_case("f32", [2] * 50, 90, 8)
    acc, tok, _ = compare((target, tokens, parents, start, u), 1)
    for i in range(50):
        assert acc[i] == int(tok[i, 0] == tokens[start[i] + 1])


def test_verify_streams_and_graphs():
    args = tree_case("bf16", [7, 9, 2], 4000, 5)
    want = run(*args, 4)
    for x, y in zip(run(*args, 4, stream=torch.cuda.Stream()), want):
        assert (x == y).all()
    target, tokens, parents, start, u = args
    acc, tok, path = torch.zeros(3, dtype=torch.int32, device=DEV), *(torch.zeros(3, 5, dtype=torch.int32, device=DEV) for _ in range(2))
    fixed = i32(tokens), i32(parents), i32(start), torch.tensor(u, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_verify_tree(acc, tok, path, target, *fixed)
        pa.pa_verify_tree(acc, tok, path, target, *fixed)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((acc, tok, path), want):
        assert (x.cpu().numpy() == y).all()


# ------------------------------------------------------------------ move of a path

def move_case(kv, counts, past, kept, layers, hk, d, bs, seed):
    rng = np.random.default_rng(seed)
    lens = [c + p for c, p in zip(counts, past)]
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 2
    perm = TR.ids(nb, seed, DEV)
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (nb, hk, bs, d) if layers is None else (layers, nb, hk, bs, d)
    raw = [torch.randint(0, 256, shape[:-1] + (d * (1 if kv == pa.PA_KV_FP8_E4M3 else 2),), generator=g, device=DEV,
                         dtype=torch.uint8) for _ in range(2)]
    k, v = (x if kv == pa.PA_KV_FP8_E4M3 else x.view(TR.CACHES[kv]) for x in raw)
    paths = [[0] + sorted(int(x) for x in rng.choice(np.arange(1, c), size=a, replace=False)) if a >= 0 else []
             for c, a in zip(counts, kept)]
    width = max(2, max(len(p) for p in paths))
    path = i32([p + [-1] * (width - len(p)) for p in paths])
    return k, v, tables, lens, [0] + np.cumsum(counts).tolist(), path, kept, paths


def moved(c, s, bs, skip=()):
    """The cache after the move, on bytes."""
    _, _, tables, lens, start, _, kept, paths = s
    before = c.view(torch.uint8)
    after = before.clone()
    for i, p in enumerate(paths):
        if i in skip:
            continue
        base = lens[i] - (start[i + 1] - start[i])
        for j, node in enumerate(p):
            src, dst = base + node, base + j
            after[..., int(tables[i, dst // bs]), :, dst % bs, :] = before[..., int(tables[i, src // bs]), :, src % bs, :]
    return after


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("layers,hk,d,bs", [(None, 8, 128, 16), (1, 1, 64, 8), (3, 2, 128, 32), (5, 3, 80, 16), (2, 4, 16, 1),
                                            (80, 8, 128, 5)])
def test_move_path(kv, layers, hk, d, bs):
    counts = [1, 16, 30, 5, 0, 7, 256]
    past = [3, 0, 120, 15, 9, 1000, 31]
    kept = [0, 4, 9, 4, -1, 0, 200]
    s = move_case(kv, counts, past, kept, layers, hk, d, bs, seed=hk + d)
    k, v, tables, lens, start, path, _, _ = s
    want = [moved(c, s, bs) for c in (k, v)]
    pa.pa_kv_move_path(k, v, tables, i32(lens), i32(start), path, i32(kept))
    torch.cuda.synchronize()
    for c, w in zip((k, v), want):
        assert torch.equal(c.view(torch.uint8), w)


def test_move_leaves_bad_sequences_alone():
    counts, past, kept = [6] * 9, [20] * 9, [3] * 9
    s = move_case(pa.PA_KV_F16, counts, past, kept, 2, 2, 64, 8, seed=1)
    k, v, tables, lens, start, path, _, paths = s
    path[0, 2] = path[0, 1]                  # does not rise
    path[1, 0] = 1                           # does not begin with node 0
    path[2, 3] = 6                           # leaves the tree
    path[3, 1] = -1
    lens2, kept2 = list(lens), list(kept)
    lens2[4] = 5                             # fewer positions than nodes
    kept2[5] = -1
    kept2[6] = 100
    tables[7, (20 + 3) // 8] = -1            # a block on the way
    want = [moved(c, s, 8, skip=range(8)) for c in (k, v)]
    pa.pa_kv_move_path(k, v, tables, i32(lens2), i32(start), path, i32(kept2))
    torch.cuda.synchronize()
    for c, w in zip((k, v), want):
        assert torch.equal(c.view(torch.uint8), w)


def test_move_on_a_stream_and_in_a_graph():
    s = move_case(pa.PA_KV_BF16, [12, 9], [50, 7], [4, 3], None, 4, 128, 16, seed=4)
    k, v, tables, lens, start, path, kept, _ = s
    want = [moved(c, s, 16) for c in (k, v)]
    first = k.clone(), v.clone()
    args = tables, i32(lens), i32(start), path, i32(kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_kv_move_path(k, v, *args, stream=side)
    side.synchronize()
    assert all(torch.equal(c.view(torch.uint8), w) for c, w in zip((k, v), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_kv_move_path(k, v, *args)
    k.copy_(first[0]), v.copy_(first[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(c.view(torch.uint8), w) for c, w in zip((k, v), want))


def test_move_refusals():
    k, v, tables, lens, start, path, kept, _ = move_case(pa.PA_KV_F16, [6], [20], [3], 2, 2, 64, 8, seed=1)
    base = dict(k_cache=k, v_cache=v, block_tables=tables, context_lens=i32(lens), query_start=i32(start), path=path,
                accepted=i32(kept))
    for change in (dict(v_cache=v[:1]), dict(k_cache=k.float()), dict(path=path[0]), dict(path=path.long()),
                   dict(accepted=i32([1, 2])), dict(query_start=i32([0])), dict(path=path[:, :0]),
                   dict(block_tables=tables.cpu()), dict(k_cache=k[..., ::2], v_cache=v[..., ::2])):
        with pytest.raises((ValueError, pa.PAError)):
            pa.pa_kv_move_path(**{**base, **change})


# ------------------------------------------------------------------ a whole step

@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_a_step_over_trees_equals_tokens_one_by_one(kv):
    """Write with rotation by depth, attention over the tree, verification, move of the path: the cache then holds what
    writing the tokens that stand one after another leaves, bit for bit, and the nodes that stand had the attention that
    those tokens get."""
    hq, hk, d, bs, vocab = 16, 2, 128, 16, 60
    rng = np.random.default_rng(3)
    g = torch.Generator(device=DEV).manual_seed(3)
    dt = TR.ROWS[kv]
    counts, past = [9, 16, 1, 40], [100, 31, 16, 700]
    ts = [TR.random_tree(rng, c, "random") for c in counts]
    level = []
    for t in ts:
        lv = []
        for p in t:
            lv.append(0 if p < 0 else lv[p] + 1)
        level.append(lv)
    al = pa.Allocator(200, bs)
    seqs = list(range(4))
    for i in seqs:
        al.add_seq(i)
    scales = dict(k_scale=1 / 64, v_scale=1 / 32) if kv == pa.PA_KV_FP8_E4M3 else {}
    kc, vc = (torch.zeros(200, hk, bs, d, dtype=TR.CACHES[kv], device=DEV) for _ in range(2))
    inv = (10000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float64) / 64)).float()
    tokens_in, start, target, u = [], [0] + np.cumsum(counts).tolist(), None, rng.random(sum(counts)).astype(np.float32)

    def new(n):
        return torch.randn(n, hq, d, generator=g, device=DEV).to(dt), *(
            torch.randn(n, hk, d, generator=g, device=DEV).to(dt) for _ in range(2))

    def put(k, v, q, positions, slots, caches):
        out = torch.empty_like(q)
        pa.pa_kv_write_rope(k, v, i32(positions), inv, torch.as_tensor(np.asarray(slots), device=DEV), *caches, query=q,
                            query_out=out, **scales)
        return out
    # the context
    slots, _ = al.append(seqs, past)
    q, k, v = new(sum(past))
    put(k, v, q, [p for n in past for p in range(n)], slots, (kc, vc))
    # the tree: a draft's position is its depth's, its slot the next free one
    slots, _ = al.append(seqs, counts)
    tables, lens = al.block_tables(seqs, 60)
    tables_d, lens_d = torch.from_numpy(tables).to(DEV), torch.from_numpy(lens).to(DEV)
    assert lens.tolist() == [a + b for a, b in zip(past, counts)]
    before = kc.clone(), vc.clone()
    q, k, v = new(sum(counts))
    turned = put(k, v, q, [past[i] + x for i in seqs for x in level[i]], slots, (kc, vc))
    parents = i32([p for t in ts for p in t])
    out = torch.empty_like(turned)
    most = int(lens.max())
    ws = torch.empty(pa.pa_attention_tree_workspace_size(4, sum(counts), hq, hk, d, most), dtype=torch.uint8, device=DEV)
    pa.pa_attention_tree(out, turned, kc, vc, tables_d, lens_d, i32(start), parents, d ** -0.5, most, ws, **scales)
    # targets under which some drafts stand
    p = torch.softmax(torch.randn(sum(counts), vocab, generator=g, device=DEV), 1)
    tokens = [int(x) for x in rng.integers(0, vocab, sum(counts))]
    for i, t in enumerate(ts):
        for j, parent in enumerate(t):
            if parent >= 0:
                p[start[i] + parent, tokens[start[i] + j]] += 0.8
    depth = 12
    acc = torch.empty(4, dtype=torch.int32, device=DEV)
    tok, path = (torch.empty(4, depth + 1, dtype=torch.int32, device=DEV) for _ in range(2))
    pa.pa_verify_tree(acc, tok, path, p, i32(tokens), parents, i32(start), torch.tensor(u, device=DEV))
    pa.pa_kv_move_path(kc, vc, tables_d, lens_d, i32(start), path, acc)
    torch.cuda.synchronize()
    accepted, path = acc.tolist(), path.tolist()
    assert max(accepted) >= 2
    # the same tokens one by one, into a cache as it was before the tree
    ref = before
    for i in seqs:
        rows = [start[i] + x for x in path[i][:accepted[i] + 1]]
        n = len(rows)
        at = [past[i] + j for j in range(n)]
        where = [int(tables[i, x // bs]) * bs + x % bs for x in at]
        put(k[rows], v[rows], q[rows], at, where, ref)
        blk, off = torch.tensor([x // bs for x in where], device=DEV), torch.tensor([x % bs for x in where], device=DEV)
        for c, r in zip((kc, vc), ref):
            assert torch.equal(c[blk, :, off], r[blk, :, off])
        # attention of the accepted nodes = causal attention over the moved rows
        got = torch.empty(n, hq, d, dtype=dt, device=DEV)
        ws2 = torch.empty(pa.pa_attention_causal_workspace_size(1, n, hq, hk, d, most), dtype=torch.uint8, device=DEV)
        pa.pa_attention_causal_typed(got, turned[rows].contiguous(), kc, vc, tables_d[i:i + 1], i32([past[i] + n]),
                                     i32([0, n]), d ** -0.5, most, ws2, **scales)
        kk = TR.cached(kc, tables_d[i], past[i] + n, bs, scales.get("k_scale", 1.0))
        vv = TR.cached(vc, tables_d[i], past[i] + n, bs, scales.get("v_scale", 1.0))
        sees = torch.arange(past[i] + n, device=DEV) <= past[i] + torch.arange(n, device=DEV).view(n, 1)
        want, bound = TR.tree_attention(turned[rows], kk, vv, sees, d ** -0.5, dt)
        for x in (out[rows], got):
            assert ((x.double() - want).abs() <= bound).all()


def test_caches_of_float8_tensors_and_empty_calls():
    # one-byte caches may be torch's own type; nothing to do is no error
    f8 = torch.float8_e4m3fn
    k, v = (torch.zeros(6, 2, 16, 128, dtype=f8, device=DEV) for _ in range(2))
    key = torch.randn(20, 2, 128, device=DEV, dtype=torch.float16)
    q, pos, inv = torch.randn(20, 4, 128, device=DEV, dtype=torch.float16), i32(list(range(20))), torch.ones(64, device=DEV)
    slots = torch.arange(20, device=DEV)
    u = [torch.zeros(6, 2, 16, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = []
    for caches in ((k, v), u):
        out = torch.empty_like(q)
        pa.pa_kv_write_rope(key, key, pos, inv, slots, *caches, query=q, query_out=out, k_scale=0.01, v_scale=0.01)
        att, ws = torch.empty_like(q[:3]), torch.empty(pa.pa_attention_tree_workspace_size(1, 3, 4, 2, 128, 20),
                                                       dtype=torch.uint8, device=DEV)
        pa.pa_attention_tree(att, out[17:].contiguous(), *caches, i32([[0, 1]]), i32([20]), i32([0, 3]), i32([-1, 0, 0]), 0.1, 20,
                             ws, k_scale=0.01, v_scale=0.01)
        pa.pa_kv_move_path(*caches, i32([[0, 1]]), i32([20]), i32([0, 3]), i32([[0, 2]]), i32([1]))
        outs.append((att, *(c.view(torch.uint8) for c in caches)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(u[0][1, :, 2], u[0][1, :, 3]) and u[0][1, :, 2].any()
    none = slots[:0]
    pa.pa_kv_write_rope(key[:0], key[:0], pos[:0], inv, none, k, v, query=q[:0])
    pa.pa_kv_move_path(k, v, i32([[0]])[:0], i32([]), i32([0]), i32([[0, 0]])[:0], i32([]))
    acc, tok = i32([5, 5]), i32([[5], [5]])
    pa.pa_verify_tree(acc, tok, tok.clone(), torch.zeros(0, 9, device=DEV), i32([]), i32([]), i32([0, 0, 0]),
                      torch.zeros(0, device=DEV))
    torch.cuda.synchronize()
    assert acc.tolist() == [-1, -1] and tok.tolist() == [[-1], [-1]]


# ------------------------------------------------------------------ PA_DEBUG_VALIDATE

def test_debug_validation_of_the_tree_calls():
    code = textwrap.dedent("""
        import sys, torch
        sys.path.insert(0, %r)
        import paged_kv_cache_12_gb300 as pa
        t = lambda v, d=torch.int32: torch.tensor(v, dtype=d, device="cuda")
        zeros = lambda *s, d=torch.float16: torch.zeros(s, dtype=d, device="cuda")
        codes = []

        def rc(f):
            try:
                f()
                codes.append(0)
            except pa.PAError as e:
                codes.append(e.code)
        k, v = zeros(8, 2, 16, 64), zeros(8, 2, 16, 64)
        inv, pos = torch.ones(32, device="cuda"), t([[0, 1, 2]])
        for slots, axis in (([5, 9, 5], 0), ([5, 9, 128], 0), ([5, -1, 9], 1), ([5, -1, 9], -1), ([5, -1, 9], 0)):
            rc(lambda: pa.pa_kv_write_rope(zeros(3, 2, 64), zeros(3, 2, 64), pos, inv, t(slots, torch.int64), k, v,
                                           pair_axis=t([axis] * 32)))
        ws = torch.empty(pa.pa_attention_tree_workspace_size(2, 5, 4, 2, 64, 50), dtype=torch.uint8, device="cuda")
        q, out, tab = zeros(5, 4, 64), zeros(5, 4, 64), [[0, 1, 2, 3], [4, 5, 6, 7]]
        good = dict(tab=tab, lens=[40, 33], start=[0, 3, 5], parents=[-1, 0, 0, -1, 0])
        for change in (dict(tab=[[0, 1, 9, 3], tab[1]]), dict(tab=[tab[0], [-1, 5, 6, 7]]), dict(lens=[51, 33]),
                       dict(lens=[2, 33]), dict(lens=[-1, 33]), dict(start=[0, 3, 4]), dict(start=[0, 6, 5]),
                       dict(parents=[-1, 0, 2, -1, 0]), dict(parents=[-1, 0, 0, -1, -2]), dict(), dict(tab=[[0, 1, 2, 99], tab[1]])):
            c = {**good, **change}
            rc(lambda: pa.pa_attention_tree(out, q, k, v, t(c["tab"]), t(c["lens"]), t(c["start"]), t(c["parents"]), 0.1, 50, ws))
        p, u = torch.ones(5, 9, device="cuda"), torch.zeros(5, device="cuda")
        acc, tok, path = zeros(2, d=torch.int32), zeros(2, 3, d=torch.int32), zeros(2, 3, d=torch.int32)
        for start in ([0, 3, 4], [0, 6, 5], [0, 3, 5]):
            rc(lambda: pa.pa_verify_tree(acc, tok, path, p, t([0, 1, 2, 0, 1]), t(good["parents"]), t(start), u))
        good = dict(tab=tab, lens=[40, 33], start=[0, 3, 5], path=[[0, 2], [0, -1]], acc=[1, 0])
        for change in (dict(acc=[2, 0]), dict(path=[[0, 0], [0, -1]]), dict(path=[[1, 2], [0, -1]]), dict(path=[[0, 3], [0, -1]]),
                       dict(lens=[2, 33]), dict(tab=[[0, 1, -1, 3], tab[1]]), dict(start=[1, 3, 5]), dict(), dict(acc=[0, 0])):
            c = {**good, **change}
            rc(lambda: pa.pa_kv_move_path(k, v, t(c["tab"]), t(c["lens"]), t(c["start"]), t(c["path"]), t(c["acc"])))
        print(" ".join(map(str, codes)))
    """ % os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    env = dict(os.environ, PA_DEBUG_VALIDATE="1")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=300)
    assert res.returncode == 0, res.stderr
    codes, E = [int(x) for x in res.stdout.split()], pa.PA_ERR_INVALID_ARG
    assert codes[:5] == [E, E, E, E, 0]
    assert codes[5:16] == [E] * 9 + [0, 0]
    assert codes[16:19] == [E, E, 0]
    assert codes[19:] == [E] * 7 + [0, 0]
