"""Calls of the step over a tree that the other tests do not make: block ids out of
range in every place of a tile, infinite keys, row offsets whose difference wraps."""
import math

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
