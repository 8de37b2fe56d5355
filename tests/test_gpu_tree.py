"""pa_attention_tree against attention in 64 bits (bounds derived in tree_ref.tree_attention)."""
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
KS, VS = 1 / 50.0, 1 / 30.0


def case(kv, lens, trees, hq, hk, d, bs, seed=0, grow=0.0, spare=2):
    """Inputs of a step; slots that hold no token are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + spare
    perm = TR.ids(nb, seed, DEV)
    mb = max(need) + 1
    tables = torch.full((len(lens), mb), -1, dtype=torch.int32, device=DEV)
    at = 0
    shape = (nb, hk, bs, d)
    if kv == pa.PA_KV_FP8_E4M3:
        k, v = (torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(2))
        k, v = (torch.where((c & 127) >= 0x60, c & 0x9f, c) for c in (k, v))   # magnitudes below 32
        hole = 0x7f
    else:
        k, v = (torch.randn(shape, generator=g, device=DEV).to(TR.CACHES[kv]) for _ in range(2))
        hole = float("nan")
    used = torch.zeros(nb, bs, dtype=torch.bool, device=DEV)
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
        pos = torch.arange(lens[i], device=DEV)
        used[tables[i].long()[pos // bs], pos % bs] = True
    for c in (k, v):
        c.transpose(1, 2)[~used] = hole
    counts = [len(t) for t in trees]
    nq = sum(counts)
    q = torch.randn(nq, hq, d, generator=g, device=DEV)
    if grow:   # rows whose scores rise along the context
        q = q * (1 + grow * torch.rand(nq, hq, 1, generator=g, device=DEV))
    return {"kv": kv, "k": k, "v": v, "q": q.to(TR.ROWS[kv]), "tables": tables, "lens": lens, "trees": trees, "bs": bs,
            "start": [0] + np.cumsum(counts).tolist(), "scale": d ** -0.5, "max_len": max(lens + [1])}


def workspace(s, lens=None):
    nq, hq, d = s["q"].shape
    size = pa.pa_attention_tree_workspace_size(len(s["lens"]), nq, hq, s["k"].shape[1], d, s["max_len"])
    return torch.full((size,), 0xAB, dtype=torch.uint8, device=DEV)   # needs no initialisation


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(s, ws=None, out=None, stream=None, **change):
    t = {**s, **change}
    ws = workspace(s) if ws is None else ws
    out = torch.full_like(s["q"], 9.0) if out is None else out
    parents = t.get("parents", [p for tree in t["trees"] for p in tree])
    scales = dict(k_scale=KS, v_scale=VS) if s["kv"] == pa.PA_KV_FP8_E4M3 else {}
    pa.pa_attention_tree(out, t["q"], t["k"], t["v"], t["tables"], i32(t["lens"]), i32(t["start"]), i32(parents),
                         t["scale"], t["max_len"], ws, stream=stream, **scales)
    torch.cuda.synchronize()
    assert pa.pa_workspace_status(ws) == pa.PA_OK
    return out


def unit(kv, x):
    return x if kv == pa.PA_KV_FP8_E4M3 else 1.0


def check(s, out, skip=(), only=None):
    """Every row against the 64-bit form (`skip`: sequences not looked at)."""
    for i, (n, tree) in enumerate(zip(s["lens"], s["trees"])):
        if i in skip or not tree:
            continue
        r = slice(s["start"][i], s["start"][i + 1])
        k = TR.cached(s["k"], s["tables"][i], n, s["bs"], unit(s["kv"], KS))
        v = TR.cached(s["v"], s["tables"][i], n, s["bs"], unit(s["kv"], VS))
        T = len(tree)
        sees = torch.ones(T, n, dtype=torch.bool)
        sees[:, n - T:] = TR.ancestors(tree)
        want, bound = TR.tree_attention(s["q"][r], k, v, sees.to(DEV), s["scale"], TR.ROWS[s["kv"]])
        off = (out[r].double() - want).abs()
        assert (off <= bound).all(), (i, float((off / bound).max()))


def trees(counts, seed=0):
    rng = np.random.default_rng(seed)
    return [TR.random_tree(rng, n, TR.KINDS[i % 5]) if n else [] for i, n in enumerate(counts)]


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("hq,hk,d,bs", [(64, 8, 128, 16), (8, 8, 128, 32), (10, 2, 128, 8), (16, 1, 128, 16), (12, 4, 64, 8),
                                        (64, 8, 64, 16), (3, 1, 64, 32), (14, 2, 128, 16)])
def test_ragged_batch(kv, hq, hk, d, bs):
    if kv == pa.PA_KV_FP8_E4M3 and d != 128:
        pytest.skip("FP8 caches have head_dim 128")
    counts = [1, 8, 3, 17, 33, 0, 5, 64, 2]
    past = [0, 0, 1, 120, 128, 40, 700, 300, 1500]
    s = case(kv, [c + p for c, p in zip(counts, past)], trees(counts, hq), hq, hk, d, bs, seed=hq + d)
    check(s, run(s))


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 127, 128, 129, 200, 255, 256])
def test_tree_sizes(kv, T):
    kinds = [[TR.random_tree(np.random.default_rng(T), T, k)] for k in ("random", "chain")]
    for past, tree in ((T % 131, kinds[0]), (300 - T, kinds[1])):
        past = max(0, past)
        s = case(kv, [T + past], tree, 8, 2, 128, 16, seed=T)
        check(s, run(s))


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("hq,hk,counts,past", [(8, 1, [16], [20000]), (64, 8, [40, 7], [9000, 40]), (16, 2, [64], [4097]),
                                               (32, 32, [3, 4], [5000, 2500])])
def test_long_contexts_cut_into_pieces(kv, hq, hk, counts, past):
    s = case(kv, [c + p for c, p in zip(counts, past)], trees(counts, 3), hq, hk, 128, 16, seed=past[0])
    check(s, run(s))


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_many_short_sequences(kv):
    rng = np.random.default_rng(4)
    counts = [int(x) for x in rng.integers(0, 9, 300)]
    past = [int(x) for x in rng.integers(0, 40, 300)]
    s = case(kv, [c + p for c, p in zip(counts, past)], trees(counts, 6), 8, 2, 128, 16, seed=17)
    check(s, run(s))


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_a_chain_is_causal_attention(kv):
    counts = [4, 4, 1, 20]
    s = case(kv, [300, 57, 1000, 420], [TR.random_tree(None, n, "chain") for n in counts], 16, 2, 128, 16, seed=3)
    out = run(s)
    nq, hq, d = s["q"].shape
    ws = torch.zeros(pa.pa_attention_causal_workspace_size(4, nq, hq, 2, d, 1000), dtype=torch.uint8, device=DEV)
    want = torch.empty_like(out)
    scales = dict(k_scale=KS, v_scale=VS) if kv == pa.PA_KV_FP8_E4M3 else {}
    pa.pa_attention_causal_typed(want, s["q"], s["k"], s["v"], s["tables"], i32(s["lens"]), i32(s["start"]), s["scale"],
                                 1000, ws, **scales)
    torch.cuda.synchronize()
    check(s, out)
    check(s, want)   # both are within the bound of the same 64-bit rows


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_running_maximum_grows_for_some_rows(kv):
    # keys far along the context that single rows score highly, so that a row's
    # maximum jumps while its neighbours' stay
    counts, hq, hk, d = [24, 40], 8, 2, 128
    s = case(kv, [1500, 900], trees(counts, 9), hq, hk, d, 16, seed=23)
    for i, (row, pos) in enumerate([(3, 400), (10, 700), (17, 1100), (30, 600), (50, 850)]):
        seq = 0 if row < 24 else 1
        blk, off = int(s["tables"][seq, pos // 16]), pos % 16
        key = s["q"][row, i % hq].float() * 3.0
        if kv == pa.PA_KV_FP8_E4M3:
            key = (key / KS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k"][blk, (i % hq) * hk // hq, off] = key.to(s["k"].dtype)
    check(s, run(s))


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("T,past,hq", [(9, 100, 8), (40, 120, 8), (130, 60, 8), (40, 3, 16)])
def test_what_a_node_does_not_see_may_be_anything(kv, T, past, hq):
    rng = np.random.default_rng(T)
    tree = TR.random_tree(rng, T, "random")
    s = case(kv, [T + past, 50], [tree, [-1, 0]], hq, 1, 128, 16, seed=T)
    sees = TR.ancestors(tree)
    good = run(s).clone()
    # poison the keys and values of two nodes: rows that do not see them keep their bits
    for what in ("k", "v", "both"):
        t = dict(s, k=s["k"].clone(), v=s["v"].clone())
        bad = [T // 2, T - 1]
        for b, x in zip(bad, (float("nan"), float("inf"))):
            pos = past + b
            for name in ("k", "v") if what == "both" else (what,):
                c = t[name]
                c[int(s["tables"][0, pos // 16]), :, pos % 16, 3] = 0x7f if kv == pa.PA_KV_FP8_E4M3 else x
        out = run(t)
        hit = torch.zeros(T + 2, dtype=torch.bool)
        hit[:T] = sees[:, bad].any(1)
        if what == "k" and kv != pa.PA_KV_FP8_E4M3:
            hit[:T] = sees[:, bad[0]]   # an infinite key may score minus infinity: only NaN is sure
            keep = ~sees[:, bad].any(1)
        else:
            keep = ~hit[:T]
        keep = torch.cat([keep, torch.ones(2, dtype=torch.bool)])
        assert torch.equal(out[keep.to(DEV)], good[keep.to(DEV)]), what
        assert (~torch.isfinite(out[hit.to(DEV)])).any(dim=-1).all(), what


def test_invalid_sequences_get_nan_rows():
    counts = [4, 5, 6, 3, 7, 2]
    tr = trees(counts, 1)
    lens = [40, 50, 60, 30, 70, 20]
    s = case(pa.PA_KV_F16, lens, tr, 8, 2, 128, 16, seed=2)
    good = run(s).clone()

    def only(bad, out):
        for i in range(6):
            r = slice(s["start"][i], s["start"][i + 1])
            if i in bad:
                assert torch.isnan(out[r]).all(), i
            else:
                assert torch.equal(out[r], good[r]), i
    only([1], run(s, lens=lens[:1] + [-1] + lens[2:]))
    only([0, 4], run(s, lens=[71] + lens[1:4] + [71] + lens[5:]))            # past max_context_len
    only([3], run(s, lens=lens[:3] + [2] + lens[4:]))                        # more nodes than positions
    tab = s["tables"].clone()
    tab[2, 1], tab[5, 0] = s["k"].shape[0], -7
    only([2, 5], run(s, tables=tab))
    tab = s["tables"].clone()
    tab[:, -1] = 1 << 30                                                     # behind every context: not looked at
    only([], run(s, tables=tab))
    st = list(s["start"])
    st[2] = st[3] + 1
    assert torch.isnan(run(s, start=st)).all()
    assert torch.isnan(run(s, start=s["start"][:-1] + [s["start"][-1] - 1])).all()
    assert torch.isnan(run(s, start=[1] + s["start"][1:])).all()


def test_bad_parents_make_their_rows_nan():
    s = case(pa.PA_KV_BF16, [60, 40], [TR.random_tree(None, 8, "chain"), [-1, 0, 0]], 8, 1, 128, 16, seed=2)
    good = run(s).clone()
    for node, parent in ((3, 3), (3, 7), (3, -2), (3, 1 << 30), (3, -(1 << 31)), (0, 0)):
        p = [p for t in s["trees"] for p in t]
        p[node] = parent
        out = run(s, parents=p)
        assert torch.isnan(out[node:8]).all() and torch.equal(out[:node], good[:node])
        assert torch.equal(out[8:], good[8:])


def test_too_many_nodes():
    T = pa.PA_TREE_MAX_NODES + 1
    s = case(pa.PA_KV_F16, [T + 5, 30], [TR.random_tree(None, T, "chain"), [-1, 0, 0]], 2, 1, 64, 8, seed=2)
    out = run(s)
    assert torch.isnan(out[:T]).all()
    check(s, out, skip=(0,))


def test_only_invalid_or_empty_sequences():
    s = case(pa.PA_KV_F16, [8, 0], [TR.random_tree(None, 8, "chain"), []], 2, 1, 64, 8, seed=2)
    assert torch.isnan(run(s, lens=[-3, 0])).all()
    out = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    t = dict(s, q=out, start=[0, 0, 0], trees=[[], []])
    pa.pa_attention_tree(out, out, s["k"], s["v"], s["tables"], i32([8, 0]), i32([0, 0, 0]), i32([]), 0.1, 8, workspace(t))


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_placement_does_not_matter_and_calls_repeat(kv):
    counts = [20, 9, 33]
    s = case(kv, [2000, 300, 1400], trees(counts, 2), 16, 2, 128, 16, seed=6)
    ws = workspace(s)
    first = run(s, ws).clone()
    nb = s["k"].shape[0]
    perm = TR.ids(nb, 99, DEV).long()
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(nb, device=DEV)
    moved = dict(s, k=s["k"][perm], v=s["v"][perm],
                 tables=torch.where(s["tables"] >= 0, inv[s["tables"].clamp(min=0).long()].int(), -1))
    for _ in range(3):
        assert torch.equal(run(moved, ws), first)


def test_streams_and_captured_calls():
    a = case(pa.PA_KV_BF16, [3000, 50], trees([20, 4], 2), 16, 2, 128, 16, seed=6)
    b = case(pa.PA_KV_F16, [700, 1200], trees([40, 30], 3), 8, 8, 64, 16, seed=7)
    wants = [run(a).clone(), run(b).clone()]
    sides = [torch.cuda.Stream() for _ in range(2)]
    wss, outs = [workspace(a), workspace(b)], [torch.zeros_like(a["q"]), torch.zeros_like(b["q"])]
    arrays = [(i32(s["lens"]), i32(s["start"]), i32([p for t in s["trees"] for p in t])) for s in (a, b)]

    def enqueue(j, stream=None):
        s = (a, b)[j]
        pa.pa_attention_tree(outs[j], s["q"], s["k"], s["v"], s["tables"], arrays[j][0], arrays[j][1], arrays[j][2],
                             s["scale"], s["max_len"], wss[j], stream=stream)
    torch.cuda.synchronize()
    for j in (0, 1):   # two calls at once
        enqueue(j, sides[j])
    torch.cuda.synchronize()
    for j in (0, 1):
        assert torch.equal(outs[j], wants[j])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):   # one after the other, over one workspace
        big = max(wss, key=lambda w: w.numel())
        wss[:] = [big, big]
        enqueue(0), enqueue(1)
    for _ in range(2):
        outs[0].zero_(), outs[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for j in (0, 1):
            assert torch.equal(outs[j], wants[j])


def test_cache_beyond_32_bits():
    # a cache of more than 2^31 elements: blocks at its far end
    nb, hk, bs, d = 70000, 8, 32, 128
    k, v = (torch.empty(nb, hk, bs, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    s = case(pa.PA_KV_BF16, [500, 77], trees([16, 5], 5), 64, hk, d, bs, seed=8)
    old = s["k"].shape[0]
    k[nb - old:], v[nb - old:] = s["k"], s["v"]
    want = run(s).clone()
    far = dict(s, k=k, v=v, tables=torch.where(s["tables"] >= 0, s["tables"] + (nb - old), -1))
    assert torch.equal(run(far), want)


def test_refusals():
    s = case(pa.PA_KV_F16, [40, 20], [[-1, 0, 0], [-1]], 8, 2, 128, 16, seed=1)
    base = dict(out=torch.empty_like(s["q"]), query=s["q"], k_cache=s["k"], v_cache=s["v"], block_tables=s["tables"],
                context_lens=i32(s["lens"]), query_start=i32(s["start"]), parents=i32([-1, 0, 0, -1]), scale=0.1,
                max_context_len=40, workspace=workspace(s))
    pa.pa_attention_tree(**base)

    def refused(**change):
        with pytest.raises((ValueError, pa.PAError)):
            pa.pa_attention_tree(**{**base, **change})
    refused(out=base["out"].bfloat16())
    refused(query=s["q"][:, :7])
    refused(query=s["q"][..., :64])
    refused(out=base["out"][:3])
    refused(k_cache=s["k"].float())
    refused(v_cache=s["v"][:-1])
    refused(parents=base["parents"][:3])
    refused(parents=base["parents"].long())
    refused(query_start=base["query_start"][:2])
    refused(context_lens=base["context_lens"][:1])
    refused(scale=0.0)
    refused(scale=float("nan"))
    refused(max_context_len=-1)
    refused(workspace=base["workspace"][:100])
    refused(workspace=base["workspace"].cpu())
    refused(k_cache=s["k"].view(torch.uint8)[..., :64].contiguous(), v_cache=s["v"].view(torch.uint8)[..., :64].contiguous())


def test_pieces_of_one_and_two_halves_in_one_range():
    # row tiles of more than 128 rows between shorter ones, several of them a CTA, cut
    # or not, in an order that gives every CTA both kinds; with infinities and NaN in
    # the values of nodes that are no ancestors
    rng = np.random.default_rng(12)
    counts = [int(x) for x in rng.choice([1, 3, 16, 17, 20, 33, 48, 64], 90)]
    past = [int(x) for x in rng.integers(0, 700, 90)]
    s = case(pa.PA_KV_BF16, [c + p for c, p in zip(counts, past)], trees(counts, 5), 64, 8, 128, 16, seed=31)
    out = run(s)
    check(s, out)
    for i in range(0, 90, 7):   # a leaf of every seventh tree
        leaf, pos = counts[i] - 1, past[i] + counts[i] - 1
        s["v"][int(s["tables"][i, pos // 16]), :, pos % 16, 9] = float("nan" if i % 2 else "inf")
        row = s["start"][i] + leaf
        out[row] = float("nan")
    again = run(s)
    nan = torch.isnan(out).all(dim=-1)
    assert torch.equal(again[~nan], out[~nan])
    assert (~torch.isfinite(again[nan])).any(dim=-1).all()


def test_waits_that_run_out():
    # PA_WAIT_LIMIT_CYCLES (read once, so in a process of its own) at one clock: a
    # wait that is not over when it first returns gives up.  A call either comes out
    # as usual, or reports PA_ERR_TIMEOUT with NaN in every row; the context is
    # usable after each
    code = textwrap.dedent("""
        import sys, numpy as np, torch
        sys.path[:0] = [%r, %r]
        import latent_ref as R
        import paged_kv_cache_12_gb300 as pa
        import test_gpu_tree as TT
        seen = []
        for kv in R.KVS:
            for hq, hk in ((8, 2), (64, 8)):
                counts = [5, 40, 1, 17, 64]
                s = TT.case(kv, [c + p for c, p in zip(counts, [3000, 100, 0, 900, 5000])], TT.trees(counts), hq, hk, 128, 16)
                ws = TT.workspace(s)
                for _ in range(3):
                    out = torch.zeros_like(s["q"])
                    scales = dict(k_scale=TT.KS, v_scale=TT.VS) if kv == pa.PA_KV_FP8_E4M3 else {}
                    pa.pa_attention_tree(out, s["q"], s["k"], s["v"], s["tables"], TT.i32(s["lens"]), TT.i32(s["start"]),
                                         TT.i32([p for t in s["trees"] for p in t]), s["scale"], s["max_len"], ws, **scales)
                    st = pa.pa_workspace_status(ws)
                    seen.append(st)
                    if st == pa.PA_OK:
                        TT.check(s, out)
                    else:
                        assert st == pa.PA_ERR_TIMEOUT and torch.isnan(out).all(), st
        print(" ".join(map(str, seen)))
    """ % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, PA_WAIT_LIMIT_CYCLES="1"))
    assert res.returncode == 0, res.stderr
    assert pa.PA_ERR_TIMEOUT in {int(x) for x in res.stdout.split()}
