"""Calls of the step over a tree that the other tests do not make: block ids out of
range in every place of a tile, infinite keys, row offsets whose difference wraps,
negative zeros, paths of many waves, a chain beside pa_verify_drafts, captured steps."""
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

import test_gpu_tree as TT
import test_gpu_tree_verify as TV

DEV = torch.device("cuda:0")


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("nodes,hq", [(9, 8), (40, 16)])   # one half, two halves (of 16-bit caches)
def test_a_bad_block_id_in_every_place_of_a_tile(kv, bs, nodes, hq):
    # sequence i's id in place i of a tile (the first one, a middle one, the last) is out of
    # range: its rows, and no others, are NaN
    boxes, L = 128 // bs, 300
    b = boxes + 2
    s = TT.case(kv, [L] * b, TT.trees([nodes] * b, bs), hq, 2, 128, bs, seed=bs + nodes)
    good = TT.run(s).clone()
    blocks = -(-L // bs)
    for tile in range(3):
        tab, bad = s["tables"].clone(), []
        for i in range(boxes):
            at = tile * boxes + i
            if at < blocks:   # (ids behind the context are not looked at)
                tab[i, at] = (s["k"].shape[0], -1, 1 << 30)[i % 3]
                bad.append(i)
        for _ in range(3):
            out = TT.run(s, tables=tab)
            for i in range(b):
                r = slice(s["start"][i], s["start"][i + 1])
                if i in bad:
                    assert torch.isnan(out[r]).all(), (tile, i)
                else:
                    assert torch.equal(out[r], good[r]), (tile, i)


@pytest.mark.parametrize("kv", [pa.PA_KV_F16, pa.PA_KV_BF16], ids=["f16", "bf16"])   # (E4M3 has no infinities)
@pytest.mark.parametrize("hq,d", [(8, 128), (8, 64)])
@pytest.mark.parametrize("T,past", [(6, 140), (40, 90)])   # one half, two halves
@pytest.mark.parametrize("inf", [math.inf, -math.inf])
def test_infinite_keys(kv, hq, d, T, past, inf):
    # a key's infinity times a query element of its sign is a score of plus infinity and a
    # row that is not finite; of the other sign a score of minus infinity, a probability of
    # 0, and the row is the one without that position
    tree = TR.random_tree(np.random.default_rng(T), T, "random")
    s = TT.case(kv, [T + past, 50], [tree, [-1, 0]], hq, 1, d, 16, seed=T)
    sign = torch.rand(T + 2, hq, generator=torch.Generator().manual_seed(3)).to(DEV) < 0.5
    s["q"][..., 3] = torch.where(sign, 0.75, -0.75).to(s["q"].dtype)
    good = TT.run(s).clone()
    sees = torch.ones(T, T + past, dtype=torch.bool)
    sees[:, past:] = TR.ancestors(tree)
    k, v = (TR.cached(s[c], s["tables"][0], T + past, 16, 1.0) for c in ("k", "v"))
    for pos in (5, past - 1, past, past + T // 2):   # in a tile without nodes or before them, node 0, a later node
        keys = s["k"].clone()
        keys[int(s["tables"][0, pos // 16]), 0, pos % 16, 3] = inf
        out = TT.run(dict(s, k=keys))
        sees_it = sees[:, pos].to(DEV).view(T, 1)
        up = sees_it & (sign[:T] == (inf > 0))
        assert torch.isnan(out[:T][up]).all(), pos
        assert torch.equal(out[:T][~sees_it.expand(T, hq)], good[:T][~sees_it.expand(T, hq)]), pos
        assert torch.equal(out[T:], good[T:])
        rest = sees.clone()
        rest[:, pos] = False
        some = rest.any(1).to(DEV).view(T, 1)
        want, bound = TR.tree_attention(s["q"][:T], k, v, rest.to(DEV), s["scale"], TR.ROWS[kv])
        low = sees_it & ~up & some
        assert low.any() and ((out[:T].double() - want).abs() <= bound)[low].all(), pos


def test_a_row_whose_only_score_is_minus_infinity_is_nan():
    s = TT.case(pa.PA_KV_F16, [1], [[-1]], 2, 1, 64, 8, seed=1)
    s["q"][0, :, 3] = torch.tensor([0.5, -0.5], dtype=torch.float16, device=DEV)
    s["k"][int(s["tables"][0, 0]), 0, 0, 3] = math.inf
    assert torch.isnan(TT.run(s)).all()


# ------------------------------------------------------------------ move of a path

def test_a_path_stays_where_row_offsets_lie_further_apart_than_an_int():
    # 2^31 - 1 and -2^31 + 5 differ by 6 where a difference wraps
    counts, past, kept = [6, 6], [20, 20], [3, 3]
    s = TV.move_case(pa.PA_KV_F16, counts, past, kept, 2, 2, 64, 8, seed=1)
    k, v, tables, lens, _, path, _, _ = s
    before = k.clone(), v.clone()
    for start in ([(1 << 31) - 1, -(1 << 31) + 5, 12], [0, (1 << 31) - 1, -(1 << 31) + 5], [6, 0, -6]):
        pa.pa_kv_move_path(k, v, tables, TT.i32(lens), TT.i32(start), path, TT.i32(kept))
        torch.cuda.synchronize()
        for c, w in zip((k, v), before):
            assert torch.equal(c.view(torch.uint8), w.view(torch.uint8)), start


# ------------------------------------------------------------------ verification

@pytest.mark.parametrize("kind,low", [("f32", -120), ("f16", -24), ("bf16", -120)])
@pytest.mark.parametrize("seqs,vocab", [(700, 9001), (2, 300007), (20, 20004)])
def test_negative_zeros_weigh_nothing(kind, low, seqs, vocab):
    # powers of two in rising order (each step's largest passes the sum before it) with a
    # negative zero in every second place; rows of negative zeros alone have no token.
    # The draws lie as far from their borders as in test_weights_of_many_sizes.
    rng = np.random.default_rng(seqs)
    x = np.sort(np.exp2(rng.integers(low, 1, (seqs, vocab)).astype(np.float64)), axis=1)
    x[rng.random((seqs, vocab)) < 0.5] = -0.0
    x[1::4] = -0.0
    target = torch.from_numpy(x).to(TV.TYPES[kind]).to(DEV)
    assert torch.signbit(target[1]).all()
    got = TV.compare((target, [0] * seqs, [-1] * seqs, list(range(seqs + 1)), rng.random(seqs).astype(np.float32)), 0)
    assert all((got[1][i, 0] == -1) == (i % 4 == 1) for i in range(seqs))


@pytest.mark.parametrize("kind,counts,vocab", [("bf16", [30] * 64, 5003), ("f32", [60, 45] * 20, 1200), ("f16", [90] * 3, 40009)])
def test_paths_of_many_waves(kind, counts, vocab):
    acc, _, _ = TV.compare(TV.tree_case(kind, counts, vocab, vocab, likely=0.97), max(counts))
    assert acc.max() >= 10


@pytest.mark.parametrize("behind", [1023, 1024, 1500])
def test_children_far_behind_their_parents(behind):
    # a wave takes descendants among the 1024 nodes behind the present one; the path goes on to those further behind
    n = 2 * behind + 9
    parents = [-1] + [0 if j <= behind else j - behind for j in range(1, n)]
    g = torch.Generator().manual_seed(behind)
    target = torch.softmax(torch.randn(4 * n, 3, generator=g), 1).to(DEV)
    tokens = np.random.default_rng(behind).integers(0, 3, 4 * n).tolist()
    for j in range(4 * n):   # few children of the root have a token of the vocabulary: those behind them decide
        if j % n <= behind and j % n != 1 + j // n:
            tokens[j] = -1
    u = np.random.default_rng(6).random(4 * n).astype(np.float32)
    for i in range(4):       # the root's one child, its child `behind` further on, if it is drafted
        tokens[i * n + 1 + i] = int(target[i * n].argmax())
        u[i * n] = float((target[i * n, :tokens[i * n + 1 + i]].double().sum() + 0.5 * target[i * n].max().double())
                         / target[i * n].double().sum())
        tokens[i * n + 1 + i + behind] = int(target[i * n + 1 + i].argmax())
        at = i * n + 1 + i
        u[at] = float((target[at, :tokens[at + behind]].double().sum() + 0.5 * target[at].max().double())
                      / target[at].double().sum())
    acc, _, path = TV.compare((target, tokens, parents * 4, [i * n for i in range(5)], u), 5)
    assert (acc >= 2).all() and path[:, 2].tolist() == [1 + i + behind for i in range(4)]


def test_a_draft_stands_as_often_as_pa_verify_drafts_lets_it():
    # chains of one draft of probability one, n of them with the same rows: by either call
    # the draft stands with probability p(draft) and the first token is distributed as p, the
    # second one after a draft that stands as the draft's row.  A share of m draws is within
    # five standard deviations of its probability (six of a million runs would not be).
    n, draft = 20000, 2
    rows = torch.tensor([[0.3, 0.15, 0.4, 0.1, 0.05], [0.1, 0.2, 0.3, 0.15, 0.25]])
    target = rows.repeat(n, 1).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(11)
    u = torch.rand(2 * n, generator=g, device=DEV)
    first = torch.arange(n + 1, device=DEV, dtype=torch.int32)
    acc, tok, path = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((n,), (n, 2), (n, 2)))
    pa.pa_verify_tree(acc, tok, path, target, TT.i32([0, draft] * n), TT.i32([-1, 0] * n), 2 * first, u)
    acc2, tok2 = torch.empty_like(acc), torch.empty_like(tok)
    pa.pa_verify_drafts(acc2, tok2, target, None, TT.i32([draft] * n), first, torch.rand(n, generator=g, device=DEV),
                        torch.rand(n, generator=g, device=DEV))
    torch.cuda.synchronize()

    def near(hits, m, p):
        assert abs(hits / m - p) <= 5 * math.sqrt(p * (1 - p) / m), (hits / m, p)
    for a, t in ((acc, tok), (acc2, tok2)):
        a, t = a.cpu(), t.cpu()
        near(int(a.sum()), n, float(rows[0, draft]))
        for v in range(5):
            near(int((t[:, 0] == v).sum()), n, float(rows[0, v]))
        after = t[a == 1]
        assert torch.equal(t[:, 0] == draft, a == 1) and (t[a == 0, 1] == -1).all()
        for v in range(5):
            near(int((after[:, 1] == v).sum()), len(after), float(rows[1, v]))


# ------------------------------------------------------------------ captured calls

def test_first_calls_of_a_process_may_be_captured():
    # what a call asks of the device once is asked while the stream is captured
    code = textwrap.dedent("""
        import sys, torch
        sys.path[:0] = [%r, %r]
        import latent_ref as R
        import paged_kv_cache_12_gb300 as pa
        import test_gpu_tree as TT
        import test_gpu_tree_verify as TV
        calls, outs = [], []
        for kv in R.KVS:
            s = TT.case(kv, [300, 50], TT.trees([20, 5]), 16, 2, 128, 16, seed=3)
            ws, out = TT.workspace(s), torch.zeros_like(s["q"])
            arrays = TT.i32(s["lens"]), TT.i32(s["start"]), TT.i32([p for t in s["trees"] for p in t])
            scales = dict(k_scale=TT.KS, v_scale=TT.VS) if kv == pa.PA_KV_FP8_E4M3 else {}
            calls.append(lambda s=s, ws=ws, out=out, arrays=arrays, scales=scales: pa.pa_attention_tree(
                out, s["q"], s["k"], s["v"], s["tables"], *arrays, s["scale"], s["max_len"], ws, **scales))
            outs.append(out)
        for kind in TV.TYPES:   # more than eight nodes a tree: the widest clusters
            target, tokens, parents, start, u = TV.tree_case(kind, [20, 12], 3000, 5)
            got = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((2,), (2, 9), (2, 9))]
            fixed = TT.i32(tokens), TT.i32(parents), TT.i32(start), torch.tensor(u, device="cuda")
            calls.append(lambda got=got, target=target, fixed=fixed: pa.pa_verify_tree(*got, target, *fixed))
            outs += got
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for c in calls:
                c()
        graph.replay()
        torch.cuda.synchronize()
        captured = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        for c in calls:
            c()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(captured, outs))
        print("same")
    """ % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.split()[-1:] == ["same"], res.stderr


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_a_captured_step_replayed_with_other_inputs(kv):
    """Write with rotation, attention, verification and move as one graph: each replay leaves what the calls one after
    another leave from the same inputs and caches."""
    hq, hk, d, bs, vocab, depth = 16, 2, 128, 16, 500, 8
    counts, past = [9, 16, 1, 40], [100, 31, 16, 700]
    n, start = sum(counts), [0] + np.cumsum(counts).tolist()
    dt = TR.ROWS[kv]
    lens = [a + b for a, b in zip(counts, past)]
    need = [-(-x // bs) for x in lens]
    ids = TR.ids(sum(need), 5, torch.device("cpu")).tolist()
    tables = [[ids.pop() for _ in range(x)] for x in need]
    slots = torch.tensor([t[p // bs] * bs + p % bs for t, m, x in zip(tables, past, lens) for p in range(m, x)], device=DEV)
    tables = TT.i32([t + [-1] * (max(need) - len(t)) for t in tables])
    lens_d, start_d = TT.i32(lens), TT.i32(start)
    inv = (10000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float64) / 64)).float()
    scales = dict(k_scale=1 / 64, v_scale=1 / 32) if kv == pa.PA_KV_FP8_E4M3 else {}
    g = torch.Generator(device=DEV).manual_seed(9)
    shape = (sum(need), hk, bs, d)

    def inputs(seed):
        q = torch.randn(n, hq, d, generator=g, device=DEV).to(dt)
        k, v = (torch.randn(n, hk, d, generator=g, device=DEV).to(dt) for _ in range(2))
        p, tokens, parents, _, u = TV.tree_case("bf16", counts, vocab, seed)
        level = []
        for j, up in enumerate(parents):
            first = max(x for x in start if x <= j)
            level.append(0 if up < 0 else level[first + up] + 1)
        pos = TT.i32([past[i] + level[j] for i in range(4) for j in range(start[i], start[i + 1])])
        return [q, k, v, pos, p.contiguous(), TT.i32(tokens), TT.i32(parents), torch.tensor(u, device=DEV)]

    def outputs():
        return [torch.empty(n, hq, d, dtype=dt, device=DEV), torch.empty(n, hq, d, dtype=dt, device=DEV),
                *(torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((4,), (4, depth + 1), (4, depth + 1)))]
    ws = torch.empty(pa.pa_attention_tree_workspace_size(4, n, hq, hk, d, max(lens)), dtype=torch.uint8, device=DEV)

    def step(x, y, kc, vc):
        q, k, v, pos, p, tokens, parents, u = x
        turned, out, acc, tok, path = y
        pa.pa_kv_write_rope(k, v, pos, inv, slots, kc, vc, query=q, query_out=turned, **scales)
        pa.pa_attention_tree(out, turned, kc, vc, tables, lens_d, start_d, parents, d ** -0.5, max(lens), ws, **scales)
        pa.pa_verify_tree(acc, tok, path, p, tokens, parents, start_d, u)
        pa.pa_kv_move_path(kc, vc, tables, lens_d, start_d, path, acc)
    fixed, got = inputs(1), outputs()
    kc, vc = (torch.zeros(shape, dtype=TR.CACHES[kv], device=DEV) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(fixed, got, kc, vc)
    moved = 0
    for seed in (2, 3, 4):
        x, want = inputs(seed), outputs()
        raw = [torch.randint(0, 0x60 if kv == pa.PA_KV_FP8_E4M3 else 256, shape, generator=g, device=DEV, dtype=torch.uint8)
               for _ in range(2)]
        held = [r if kv == pa.PA_KV_FP8_E4M3 else (r.float() / 64 - 2).to(dt) for r in raw]
        for a, b in zip(fixed + [kc, vc], x + held):
            a.copy_(b)
        graph.replay()
        step(x, want, *held)
        torch.cuda.synchronize()
        for a, b in zip(got + [kc, vc], want + held):
            assert torch.equal(a, b)
        assert torch.isfinite(got[1]).all()
        moved += int(got[2].sum())
    assert moved > 3
