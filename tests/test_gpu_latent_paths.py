"""Paths of the latent-cache calls that a plain call does not reach or does not
tell apart from a mistake: what each of them has to keep is said at its test.
References are plain 64-bit forms (latent_ref.py)."""
import math
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa
from test_gpu_latent import absorbed, compare_absorbed, same_bits

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


# ------------------------------------------------------------------ waits that run out

def test_waits_that_run_out():
    # PA_WAIT_LIMIT_CYCLES (read once, so in a process of its own) at one clock: a
    # wait that is not over when it first returns gives up.  A call either comes
    # out as usual, or reports PA_ERR_TIMEOUT with NaN in every row; the context
    # is usable after each, and whatever was on its way has landed before the
    # next call's kernels take the shared memory
    code = textwrap.dedent("""
        import sys, math, torch
        sys.path[:0] = [%r, %r]
        import latent_ref as R
        import paged_kv_cache_12_gb300 as pa
        from test_gpu_latent import compare_absorbed, compare_expanded, i32
        SCALE = 1 / math.sqrt(192.0)
        seen = []

        def judge(ws, out, compare):
            st = pa.pa_workspace_status(ws)
            seen.append(st)
            if st == pa.PA_OK:
                compare()
            else:
                assert st == pa.PA_ERR_TIMEOUT and torch.isnan(out).all(), st

        for kv in R.KVS:
            lens = [(977 * i) %% 4000 + 1 for i in range(60)]
            w = R.Paged(lens, 16, kv, 5, "cuda")
            for heads in (16, 128):
                n = len(lens)
                q = torch.randn(n, heads, 576, device="cuda").to(R.TYPES[kv])
                ws = torch.empty(pa.pa_latent_attention_workspace_size(n, n, heads, 4000), dtype=torch.uint8, device="cuda")
                for _ in range(3):
                    out = torch.zeros(n, heads, 512, dtype=R.TYPES[kv], device="cuda")
                    pa.pa_latent_attention(out, q, w.cache, w.tables, w.lens_t, SCALE, 4000, ws)
                    judge(ws, out, lambda: compare_absorbed(w, q, out, None))
        for dt in (torch.float16, torch.bfloat16):
            news, pasts, heads = [300, 77, 1], [900, 0, 130], 8
            nq, nk = sum(news), sum(news) + sum(pasts)
            q = torch.randn(nq, heads, 192, device="cuda").to(dt)
            up, r = torch.randn(nk, heads, 256, device="cuda").to(dt), torch.randn(nk, 64, device="cuda").to(dt)
            k, v = up[..., :128], up[..., 128:]
            qs, ks = i32([0, 300, 377, 378]), i32([0, 1200, 1277, 1408])
            ws = torch.empty(pa.pa_latent_attention_expanded_workspace_size(3, nq, heads), dtype=torch.uint8, device="cuda")
            for _ in range(3):
                out = torch.zeros(nq, heads, 128, dtype=dt, device="cuda")
                pa.pa_latent_attention_expanded(out, q, k, r, v, qs, ks, SCALE, ws)
                judge(ws, out, lambda: compare_expanded(q, k, r, v, out, news, pasts))
        print(" ".join(map(str, seen)))
    """ % (ROOT, os.path.dirname(os.path.abspath(__file__))))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, PA_WAIT_LIMIT_CYCLES="1"))
    assert res.returncode == 0, res.stderr
    assert pa.PA_ERR_TIMEOUT in {int(x) for x in res.stdout.split()}   # (all of them where this was written)
