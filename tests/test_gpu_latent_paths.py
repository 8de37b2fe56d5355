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
from test_gpu_latent import absorbed, compare_absorbed, i32, same_bits

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


# ------------------------------------------------------------------ expanded attention

@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_expanded_many_short_sequences(dt):
    # some forty short pieces a CTA, of one or both halves of a row tile, with
    # values of new tokens that are not finite in a third of the sequences: each
    # row that sees one is not finite in that element, and every other row is as
    # the definition says.  (A record of them is kept for two pieces of a half.)
    # More sequences than the CTA has threads, some of them empty
    heads, b = 2, 3001
    g = torch.Generator().manual_seed(31)
    kinds = torch.randint(5, (b,), generator=g).tolist()
    news = [(0, 1, 5 + i % 120, 129 + i % 60, 3 + i % 20)[k] for i, k in enumerate(kinds)]
    pasts = [(0, 2 + i % 9, 0, i % 140, 40 + i % 130)[k] for i, k in enumerate(kinds)]
    lens = [a + p for a, p in zip(news, pasts)]
    qs, ks = [0], [0]
    for a, n in zip(news, lens):
        qs.append(qs[-1] + a)
        ks.append(ks[-1] + n)
    q = torch.randn(qs[-1], heads, 192, generator=g).to(dt)
    up = torch.randn(ks[-1], heads, 256, generator=g).to(dt)
    r = torch.randn(ks[-1], 64, generator=g).to(dt)
    hit = {}
    for i in range(0, b, 3):
        if news[i]:
            j, h = int(torch.randint(news[i], (1,), generator=g)), i // 3 % heads
            hit[i] = (j, h)
            up[ks[i] + pasts[i] + j, h, 128 + 9] = (math.nan, math.inf)[i // 6 % 2]
    q, up, r = q.to(DEV), up.to(DEV), r.to(DEV)
    k, v = up[..., :128], up[..., 128:]
    ws = torch.full((pa.pa_latent_attention_expanded_workspace_size(b, qs[-1], heads),), 255, dtype=torch.uint8, device=DEV)
    out = torch.zeros(qs[-1], heads, 128, dtype=dt, device=DEV)
    pa.pa_latent_attention_expanded(out, q, k, r, v, i32(qs), i32(ks), SCALE, ws)
    assert pa.pa_workspace_status(ws) == pa.PA_OK
    for i in range(b):
        n, L = news[i], lens[i]
        for h in range(heads if n else 0):
            bad = hit[i][0] if i in hit and hit[i][1] == h else n
            got = out[qs[i]:qs[i + 1], h]
            assert not torch.isfinite(got[bad:, 9]).any(), (i, h)
            s, e = ks[i], ks[i] + pasts[i] + bad
            key = torch.cat([k[s:e, h], r[s:e]], 1).double()
            o, tol = attend_causal(q[qs[i]:qs[i] + bad, h].double(), key, v[s:e, h].double(), SCALE, dt)
            R.check(got[:bad], o, tol, f"sequence {i}, head {h}") if bad else None


def attend_causal(q, k, v, scale, dt):
    """R.attend for rows q of which row j sees len(k) - len(q) + j + 1 positions
    (its tolerance with the largest of their score errors and counts)."""
    n, past = k.shape[0], k.shape[0] - q.shape[0]
    hide = torch.ones(q.shape[0], n, dtype=torch.bool, device=k.device).triu(past + 1)
    p = torch.softmax((q @ k.T * scale).masked_fill(hide, -math.inf), 1)
    o, u = p @ v, R.half_step(dt)
    d = (q.abs() @ k.abs().T).amax(1, keepdim=True) * scale * q.shape[1] * 2.0 ** -24 if n else 0.0
    tol = (u + 2 * d + n * 2.0 ** -24 + 2.0 ** -20) * (p @ v.abs()) + u * o.abs()
    if dt == torch.float16 and n:
        tol = tol + n * 2.0 ** -25 * v.abs().amax(0) + 2.0 ** -25
    return o, tol


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
