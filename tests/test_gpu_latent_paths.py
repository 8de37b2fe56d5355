"""Paths of the latent-cache calls that a plain call does not reach or does not
tell apart from a mistake: what each of them has to keep is said at its test.
References are plain 64-bit forms (latent_ref.py)."""
import math

import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa
from test_gpu_latent import absorbed, compare_absorbed, same_bits

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------ absorbed attention

def test_rotary_elements_of_quantised_rows():
    # queries without a latent part, so that the rotary elements alone choose the
    # positions: a rotary element read after its staging slot was handed back (and
    # overwritten with a later row's) moves the weight to another row.  Contexts
    # enough for every CTA to pass its slots many times, the same bits every time
    lens = [(173 * i) % 900 + 1 for i in range(160)]
    w = R.Paged(lens, 16, pa.PA_KV_FP8_E4M3, 83, DEV)
    g = torch.Generator().manual_seed(83)
    q = torch.zeros(len(lens), 16, 576, dtype=torch.bfloat16)
    for i, n in enumerate(lens):
        t = torch.randint(n, (16,), generator=g)
        q[i, :, 512:] = (3 * w.rows(i)[t.to(DEV), 512:]).to(torch.bfloat16).cpu()
    q = q.to(DEV)
    _, want = absorbed(w, 16, None, 0, query=q)
    compare_absorbed(w, q, want, None)
    for _ in range(20):
        assert same_bits(absorbed(w, 16, None, 0, query=q)[1], want)
