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
from test_gpu_latent import absorbed, compare_absorbed, expanded, i32, kvs, same_bits

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


@pytest.mark.parametrize("kv,tile", [(pa.PA_KV_BF16, 64), (pa.PA_KV_FP8_E4M3, 48)], ids=["bf16", "fp8"])
def test_every_range_of_a_long_context_counts(kv, tile):
    # 5,000,001 positions, cut into a range of KV tiles for every SM.  Blocks of
    # their own lie on both sides of every cut, at the start and at the end, each
    # with its share of the weight and the only values of some size in a dim of
    # its own; everywhere else a table names 40 blocks again and again.  So a
    # range (or a part of one) that is left out or counted twice shows in its
    # dims: five times the bound at least, which the test verifies too
    bs, plain, n, cost = 64, 40, 5_000_001, 2
    ctas = torch.cuda.get_device_properties(DEV).multi_processor_count
    g = torch.Generator().manual_seed(13)
    units = -(-n // tile) + cost
    cuts = [(units * k // ctas - cost) * tile for k in range(1, ctas)]
    own = sorted({t // bs for c in cuts for t in (c - 1, c)} | {0, (n - 1) // bs})
    assert len(own) <= 512
    nb = plain + len(own)
    latent, rope = 0.02 * torch.randn(nb, bs, 512, generator=g), torch.randn(nb, bs, 64, generator=g)
    latent[plain:] = 0
    for j in range(len(own)):
        latent[plain + j, :, j] = 4 + 8 * torch.rand(bs, generator=g)
    # a score of its own that gives those blocks about half of the weight
    rope[:, :, 0] = 0
    rope[plain:, :, 0] = math.log(n / (len(own) * bs)) / (4 * SCALE)
    q = torch.cat([0.05 * torch.randn(1, 16, 512, generator=g), 0.5 * torch.randn(1, 16, 64, generator=g)], 2)
    q[..., 512] = 4
    latent, rope, q = latent.bfloat16().view(-1, 512), rope.bfloat16().view(-1, 64), q.bfloat16()
    packed = R.pack8(latent, rope) if kv == pa.PA_KV_FP8_E4M3 else torch.cat([latent, rope], 1)
    entries = torch.randint(plain, (-(-n // bs),), generator=g)
    entries[own] = plain + torch.arange(len(own))

    rows = R.rows64(packed)
    seen = torch.zeros(nb * bs, dtype=torch.float64)
    for k in range(bs):   # the last block is seen up to its remainder
        hit = entries if k < (n - 1) % bs + 1 else entries[:-1]
        seen.view(nb, bs)[:, k] = torch.bincount(hit, minlength=nb).double()
    s = (q[0].double() @ rows.T) * SCALE + torch.log(seen)
    p = torch.softmax(s, 1)
    want, mass = p @ rows[:, :512], p @ rows[:, :512].abs()
    # a probability is rounded by at most 2^-8 of itself and the output by 2^-8 of
    # it; a score's 576 additions (in 32 bits, truncated at worst) lose at most
    # 576 * 2^-23 of the sum of magnitudes, which the softmax doubles; O and l are
    # sums over a range's positions, then over at most 160 pieces
    score = 576 * 2 ** -23 * SCALE * float((q[0].double().abs() @ rows.abs().T).max())
    bound = (2 ** -8 + 2 * score + 2 * (n // ctas + 2 * tile + 160) * 2 ** -23) * mass + 2 ** -8 * want.abs()

    part = torch.zeros(16, ctas, 512, dtype=torch.float64)   # what the blocks of their own bring to each range's outputs
    t = (torch.tensor(own).view(-1, 1) * bs + torch.arange(bs)).view(-1)
    which = torch.searchsorted(torch.tensor(cuts), t, right=True)
    at = plain * bs + torch.arange(len(own) * bs)
    dim = torch.arange(len(own)).repeat_interleave(bs)
    for h in range(16):
        part[h].view(-1).index_add_(0, which * 512 + dim, p[h, at] * rows[at, dim] * (t < n))
    assert (part / bound.view(16, 1, 512)).amax(2).min() > 5

    w = 576 if kv == pa.PA_KV_BF16 else R.ROW8
    ws = torch.empty(pa.pa_latent_attention_workspace_size(1, 1, 16, n), dtype=torch.uint8, device=DEV)
    out = torch.zeros(1, 16, 512, dtype=torch.bfloat16, device=DEV)
    pa.pa_latent_attention(out, q.to(DEV), packed.view(nb, bs, w).to(DEV), entries.int()[None].to(DEV), i32([n]), SCALE, n, ws)
    assert pa.pa_workspace_status(ws) == pa.PA_OK
    worst = ((out[0].cpu().double() - want).abs() / bound).max().item()
    assert worst <= 1, worst


@kvs
@pytest.mark.parametrize("heads,news,lens", [(128, [2, 1, 4], [5000, 3000, 700]), (16, [700, 300], [900, 300]),
                                             (128, [1, 1], [2600, 7000]), (7, [200, 1, 33], [3000, 2000, 33])])
def test_absorbed_longer_contexts_and_chunks(kv, heads, news, lens):
    w = R.Paged(lens, 32, kv, 91 + heads, DEV)
    q, out = absorbed(w, heads, news, 9)
    at = 0
    for i, (n, L) in enumerate(zip(news, lens)):
        c = w.rows(i)
        for j in range(n):
            if j in (0, 1, n // 3, n // 2, n - 2, n - 1):
                vis = L - n + j + 1
                o, tol = R.attend(q[at + j].double(), c[:vis], c[:vis, :512], SCALE, R.TYPES[kv])
                R.check(out[at + j], o, tol, f"sequence {i}, new token {j}")
        assert torch.isfinite(out[at:at + n]).all()
        at += n


def test_two_streams_at_once():
    # calls on two streams, each with a workspace of its own, in flight together
    w = R.Paged([700, 33, 1500, 64], 16, pa.PA_KV_BF16, 93, DEV)
    v = R.Paged([260, 2000], 32, pa.PA_KV_FP8_E4M3, 94, DEV)
    qw, a = absorbed(w, 16, None, 1)
    qv, b = absorbed(v, 32, [3, 2], 2)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(x) for _ in range(8)] for x in (a, b)]
    ws = [torch.full((pa.pa_latent_attention_workspace_size(4, 5, 32, 2000),), 255, dtype=torch.uint8, device=DEV)
          for _ in range(2)]
    qs = i32([0, 3, 5])
    torch.cuda.synchronize()
    for i in range(8):
        pa.pa_latent_attention(outs[0][i], qw, w.cache, w.tables, w.lens_t, SCALE, 1500, ws[0], stream=sides[0])
        pa.pa_latent_attention(outs[1][i], qv, v.cache, v.tables, v.lens_t, SCALE, 2000, ws[1], query_start=qs,
                               stream=sides[1])
    torch.cuda.synchronize()
    assert all(same_bits(x, a) for x in outs[0]) and all(same_bits(x, b) for x in outs[1])


@kvs
@pytest.mark.parametrize("captured", [False, True])
def test_cache_calls_behind_one_another(kv, captured):
    # write, copy, attention and read back queued without a pause, each on what the
    # one before has just written; several steps, then against the final cache
    bs, steps, b, heads, dt = 16, 12, 5, 16, R.TYPES[kv]
    g = torch.Generator().manual_seed(95 + kv)
    width = R.ROW8 if kv == pa.PA_KV_FP8_E4M3 else 576
    rows = torch.randn(steps, b, 576, generator=g).to(dt)
    q = torch.randn(steps, b, heads, 576, generator=g).to(dt).to(DEV)
    # sequence i: tokens at slots 16 i .. (block i), copied after every step into block b + i, which the table names
    slots = (torch.arange(b) * bs + torch.arange(steps).view(-1, 1)).to(torch.int64).to(DEV)
    pairs = torch.stack([torch.arange(b), torch.arange(b) + b], 1).to(DEV)
    tab = (torch.arange(b) + b).int().view(b, 1).to(DEV)
    lens = [i32([k + 1] * b) for k in range(steps)]
    starts = [i32([(k + 1) * i for i in range(b + 1)]) for k in range(steps)]
    cache = torch.zeros(2 * b, bs, width, dtype=torch.uint8 if kv == pa.PA_KV_FP8_E4M3 else dt, device=DEV)
    outs = torch.zeros(steps, b, heads, 512, dtype=dt, device=DEV)
    backs = [torch.zeros((k + 1) * b, 576, dtype=dt, device=DEV) for k in range(steps)]
    ws = torch.full((pa.pa_latent_attention_workspace_size(b, b, heads, bs),), 255, dtype=torch.uint8, device=DEV)
    dev = rows.to(DEV)

    def run():
        for k in range(steps):
            pa.pa_latent_write(dev[k, :, :512], dev[k, :, 512:], slots[k], cache)
            pa.pa_latent_block_copy(cache, pairs)
            pa.pa_latent_attention(outs[k], q[k], cache, tab, lens[k], SCALE, bs, ws)
            pa.pa_latent_read(backs[k], cache, tab, starts[k])

    def check():
        torch.cuda.synchronize()
        packed = R.pack8(rows.reshape(-1, 576)[:, :512], rows.reshape(-1, 576)[:, 512:]) if kv == pa.PA_KV_FP8_E4M3 else \
            rows.reshape(-1, 576)
        held = R.rows64(packed).view(steps, b, 576).to(DEV)
        for k in range(steps):
            assert torch.equal(backs[k].view(b, k + 1, 576).double(), held[:k + 1].transpose(0, 1))
            for i in range(b):
                c = held[:k + 1, i]
                o, tol = R.attend(q[k, i].double(), c, c[:, :512], SCALE, dt)
                R.check(outs[k, i], o, tol, f"step {k}, sequence {i}")

    if not captured:
        for _ in range(10):
            run()
        check()
        return
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        run()
    for _ in range(3):
        cache.zero_()
        outs.fill_(math.nan)
        for x in backs:
            x.fill_(math.nan)
        graph.replay()
        check()


# ------------------------------------------------------------------ read back of many sequences

@pytest.mark.parametrize("kv", [pa.PA_KV_BF16, pa.PA_KV_FP8_E4M3], ids=["bf16", "fp8"])
@pytest.mark.parametrize("b", [1023, 1024, 1025, 3000])
def test_read_of_many_sequences(kv, b):
    # row offsets are kept in shared memory up to 1024 sequences and searched in
    # global memory beyond; some sequences have no rows
    lens = [(7 * i) % 23 for i in range(b)]
    w = R.Paged(lens, 8, kv, b, DEV)
    first = [i % 5 if n > 5 else 0 for i, n in enumerate(lens)]
    counts = [n - f for n, f in zip(lens, first)]
    start = [0]
    for c in counts:
        start.append(start[-1] + c)
    slots = torch.cat([s[f:] for s, f in zip(w.seq_slots, first)]).to(DEV)
    want = R.rows64(w.cache)[slots] if kv == pa.PA_KV_FP8_E4M3 else w.cache.view(-1, 576)[slots].double()
    out = torch.full((start[-1] + 3, 576), 7.0, dtype=R.TYPES[kv], device=DEV)
    pa.pa_latent_read(out, w.cache, w.tables, i32(start), i32(first))
    assert torch.equal(out[:-3].double(), want) and (out[-3:] == 7).all()
    for at in (3, b // 2, b - 2):                            # an order broken anywhere makes every row NaN
        bad = list(start)
        bad[at] = start[at + 1] + 1
        out.fill_(7.0)
        pa.pa_latent_read(out, w.cache, w.tables, i32(bad), i32(first))
        assert torch.isnan(out).all(), at


# ------------------------------------------------------------------ expanded attention

def test_expanded_layouts():
    # keys and values head by head ([heads][tokens]), in padded rows and with
    # strides that are no multiples of one another: the same bits as contiguous
    dt, heads, news, pasts = torch.bfloat16, 3, [200, 40, 1], [60, 300, 0]
    q, k, r, v, want, (qs, ks, ws) = expanded(dt, news, pasts, heads, 37)
    nk = k.shape[0]

    def held(t, shape, view):
        x = torch.full(shape, math.nan, dtype=dt, device=DEV)
        y = view(x)
        y.copy_(t)
        assert y.shape == t.shape
        return y
    flat = [lambda x: x[:, :, :128], lambda x: x[:, :, 8:136]]
    layouts = [
        (held(k, (heads, nk, 128), lambda x: x.transpose(0, 1)), held(v, (heads, nk, 128), lambda x: x.transpose(0, 1))),
        (held(k, (heads, nk + 5, 136), lambda x: x[:, 2:-3, :128].transpose(0, 1)), held(v, (nk, heads, 136), flat[1])),
        (held(k, (nk, heads * 136 + 8), lambda x: x[:, :heads * 136].unflatten(1, (heads, 136))[:, :, :128]),
         held(v, (nk, heads, 200), flat[0])),
    ]
    for kk, vv in layouts:
        for rr in (r.contiguous(), held(r, (nk, 72), lambda x: x[:, 8:])):
            out = torch.zeros_like(want)
            pa.pa_latent_attention_expanded(out, q, kk, rr, vv, qs, ks, SCALE, ws)
            assert same_bits(out, want)



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
            if bad:
                R.check(got[:bad], o, tol, f"sequence {i}, head {h}")


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


# ------------------------------------------------------------------ PA_DEBUG_VALIDATE

def test_debug_validation_of_the_latent_calls():
    code = textwrap.dedent("""
        import sys, torch
        sys.path.insert(0, %r)
        import paged_kv_cache_12_gb300 as pa
        t = lambda v, d=torch.int32: torch.tensor(v, dtype=d, device="cuda")
        zeros = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")
        codes = []

        def rc(f):
            try:
                f()
                codes.append(0)
            except pa.PAError as e:
                codes.append(e.code)
        cache = zeros(8, 16, 576)
        for slots in ([5, 9, 5], [5, 9, 128], [5, -1, 9]):
            rc(lambda: pa.pa_latent_write(zeros(3, 512), zeros(3, 64), t(slots, torch.int64), cache))
        for pairs in ([[1, 2], [2, 3]], [[1, 3], [2, 3]], [[1, 8]], [[1, 3], [1, 4]]):
            rc(lambda: pa.pa_latent_block_copy(cache, t(pairs, torch.int64)))
        out, tab = zeros(40, 576), t([[0, 4], [1, 2]])
        for start, first, table in (([0, 20, 15], [0, 0], tab), ([0, 20, 41], [0, 0], tab), ([1, 20, 40], [0, 0], tab),
                                    ([0, 20, 40], [-1, 0], tab), ([0, 20, 40], [0, 13], tab),
                                    ([0, 20, 40], [0, 0], t([[0, 4], [1, 8]])), ([0, 20, 40], [0, 0], t([[0, -1], [1, 2]])),
                                    ([0, 16, 30], [0, 0], t([[0, -1], [1, 2]])), ([0, 20, 40], [12, 12], tab),
                                    ([0, 0, 20], [-9, 12], tab)):
            rc(lambda: pa.pa_latent_read(out, cache, table, t(start), t(first)))
        ws = zeros(pa.pa_latent_attention_workspace_size(2, 5, 4, 32), d=torch.uint8)
        for lens, start, table in (([20, 3], None, t([[0, 8], [1, 2]])), ([33, 3], None, tab), ([-1, 3], None, tab),
                                   ([20, 3], [0, 4, 3], tab), ([20, 3], [0, 1, 5], tab), ([20, 3], [0, 3, 4], tab),
                                   ([20, 3], None, tab), ([20, 3], [0, 2, 5], tab), ([20, 0], [0, 5, 5], t([[0, 4], [-1, -1]]))):
            n = 2 if start is None else 5
            rc(lambda: pa.pa_latent_attention(zeros(n, 4, 512), zeros(n, 4, 576), cache, table, t(lens), 0.1, 32, ws,
                                              query_start=None if start is None else t(start)))
        ws = zeros(pa.pa_latent_attention_expanded_workspace_size(2, 5, 4), d=torch.uint8)
        for a, b in (([0, 2, 4], [0, 4, 9]), ([0, 6, 5], [0, 4, 9]), ([0, 2, 5], [0, 4, 8]), ([0, 2, 5], [0, 10, 9]),
                     ([0, 2, 5], [0, 4, 9])):
            rc(lambda: pa.pa_latent_attention_expanded(zeros(5, 4, 128), zeros(5, 4, 192), zeros(9, 4, 128), zeros(9, 64),
                                                       zeros(9, 4, 128), t(a), t(b), 0.1, ws))
        for start in ([0, 2, 1], [1, 2, 3], [0, 2, 3]):
            rc(lambda: pa.pa_verify_drafts(t([0, 0]), t([[0] * 3] * 2), zeros(5, 9, d=torch.float32), None, t([1, 2, 3]),
                                           t(start), t([0.5] * 3, torch.float32), t([0.5] * 2, torch.float32)))
        torch.cuda.synchronize()
        print(" ".join(map(str, codes)))
    """ % ROOT)
    env = dict(os.environ, PA_DEBUG_VALIDATE="1")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=300)
    assert res.returncode == 0, res.stderr
    codes, E = [int(x) for x in res.stdout.split()], pa.PA_ERR_INVALID_ARG
    write, copy, read, attention, expanded_, verify = codes[:3], codes[3:7], codes[7:17], codes[17:26], codes[26:31], codes[31:]
    assert write == [E, E, 0] and copy == [E, E, E, 0]
    assert read == [E] * 7 + [0, 0, 0]
    assert attention == [E] * 6 + [0, 0, 0]
    assert expanded_ == [E] * 4 + [0] and verify == [E, E, 0]
