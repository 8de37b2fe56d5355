"""Calls of the step over a tree that the other tests do not make: block ids out of
range in every place of a tile."""
import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa
import tree_ref as TR

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

import test_gpu_tree as TT

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
