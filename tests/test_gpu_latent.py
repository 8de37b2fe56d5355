"""The latent cache on the GPU: rows written (copied or quantised), read back,
copied; attention over it in the absorbed form; attention in the expanded form;
and a serving run that uses them together.  References are plain 64-bit forms
(latent_ref.py)."""
import math

import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
SCALE = 1.0 / math.sqrt(192.0)
kvs = pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ write

@kvs
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("n", [1, 7, 100, 1003])
def test_write(kv, bs, n):
    g = torch.Generator().manual_seed(n + bs)
    dt = R.TYPES[kv]
    rows = (torch.randn(n, 600, generator=g) * torch.exp2(torch.randint(-20, 12, (n, 1), generator=g).float())).to(dt)
    latent, rope = rows[:, 8:520], rows[:, 528:592]         # slices, at 16-byte offsets
    nb = -(-n // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:n]
    slots[3::5] = -1
    if n > 10:
        slots[10] = nb * bs                                  # past the pool: skipped
    before = R.nan_cache(nb, bs, kv, "cpu")
    want = before.clone().view(nb * bs, -1)
    keep = [i for i, s in enumerate(slots.tolist()) if 0 <= s < nb * bs]
    want[slots[keep]] = R.pack8(latent[keep], rope[keep]) if kv == pa.PA_KV_FP8_E4M3 else \
        torch.cat([latent, rope], 1)[keep]
    cache, dev = before.to(DEV), rows.to(DEV)
    pa.pa_latent_write(dev[:, 8:520], dev[:, 528:592], slots.to(DEV), cache)
    assert same_bits(cache.cpu().view(nb * bs, -1), want)


def test_quantised_write_at_the_edges_of_its_range():
    # group maxima on and next to 448 * 2^e, zeros, subnormals, infinities, NaN
    mx = float(torch.finfo(torch.bfloat16).max)
    tops = [0.0, 448.0, 450.0, 446.0, 1.0, 1.75, 1.7578125, 2.0 ** -126, 2.0 ** -133, 2.0 ** -92, 2.0 ** -91 * 1.75,
            mx, mx / 2, 2.0 ** 127, 2.0 ** 127 * 1.75, math.inf, -math.inf, math.nan, -448.0, 3e38]
    n = len(tops)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, 512, generator=g).to(torch.bfloat16)
    for i, t in enumerate(tops):
        big = abs(t) if math.isfinite(t) else 1.0
        x[i] = (torch.rand(512, generator=g) * 2 - 1) * (0.9 * big)
        x[i, ::37] = 0.0
        x[i, 1::128] = t
    x[17, 64:96] = math.nan                                  # a group with a NaN among others
    rope = torch.randn(n, 64, generator=g).to(torch.bfloat16)
    rope[0, 0], rope[0, 1], rope[0, 2] = math.nan, math.inf, -0.0
    cache = torch.zeros(2, 16, R.ROW8, dtype=torch.uint8, device=DEV)
    slots = torch.arange(n, device=DEV)
    pa.pa_latent_write(x.to(DEV), rope.to(DEV), slots, cache)
    got, want = cache.view(32, -1)[:n].cpu(), R.pack8(x, rope)
    codes, codes_w = got[:, :512], want[:, :512]
    nan = (codes_w & 127) == 127
    assert torch.equal((codes & 127) == 127, nan)            # a NaN's sign is not specified
    assert torch.equal(codes[~nan] & 127, codes_w[~nan] & 127)
    signed = ~nan & (codes_w & 127 != 0)
    assert torch.equal(codes[signed], codes_w[signed])
    assert torch.equal(got[:, 512:], want[:, 512:])


# ------------------------------------------------------------------ read, copy

@kvs
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
def test_read(kv, bs):
    lens = [0, 1, 70, bs, bs + 1, 333, 0]
    w = R.Paged(lens, bs, kv, 11 + bs, DEV)
    counts = [0, 1, 64, bs, 1, 300, 0]
    first = [0, 0, 6, 0, bs, 33, 0]
    start = [0]
    for c in counts:
        start.append(start[-1] + c)
    n = start[-1]
    wide = torch.full((n + 5, 592), 7.0, dtype=R.TYPES[kv], device=DEV)
    pa.pa_latent_read(wide[:, :576], w.cache, w.tables, i32(start), i32(first))
    for i, (c, f) in enumerate(zip(counts, first)):
        if c:
            assert torch.equal(wide[start[i]:start[i + 1], :576].double(), w.rows(i)[f:f + c]), i
    assert (wide[n:] == 7).all() and (wide[:, 576:] == 7).all()      # rows behind the last, and the gap, untouched
    whole = torch.empty(sum(lens), 576, dtype=R.TYPES[kv], device=DEV)
    at = [sum(lens[:i]) for i in range(len(lens) + 1)]
    pa.pa_latent_read(whole, w.cache, w.tables, i32(at))
    assert torch.equal(whole.double(), torch.cat([w.rows(i) for i in range(len(lens))]))


@kvs
def test_read_of_bad_rows(kv):
    w = R.Paged([40, 40], 16, kv, 3, DEV)
    out = torch.zeros(80, 576, dtype=R.TYPES[kv], device=DEV)
    tab = w.tables.clone()
    tab[0, 1], tab[1, 2] = w.nb, -5
    pa.pa_latent_read(out, w.cache, tab, i32([0, 40, 80]), i32([0, 12]))
    bad = torch.zeros(80, dtype=torch.bool)
    bad[16:32] = True                                        # the block past the pool
    bad[40 + 32 - 12:] = True                                # block -5, and tokens past the table
    assert torch.equal(torch.isnan(out).all(1).cpu(), bad) and torch.equal(torch.isnan(out).any(1).cpu(), bad)
    assert torch.equal(out[:16].double(), w.rows(0)[:16])
    for start in ([0, 50, 40], [3, 40, 80], [0, 40, 81], [0, -1, 80]):
        out.zero_()
        pa.pa_latent_read(out, w.cache, w.tables, i32(start))
        assert torch.isnan(out).all(), start
    out.zero_()
    pa.pa_latent_read(out[:20], w.cache, w.tables, i32([0, 20, 20]), i32([-30, 0]))
    assert torch.isnan(out[:20]).all()


@kvs
def test_block_copy(kv):
    w = R.Paged([200], 8, kv, 9, DEV, spare=6)
    used = w.tables_np[0].tolist()
    free = [b for b in range(w.nb) if b not in used]
    want = w.cache.clone()
    pairs = [(used[0], free[0]), (used[0], free[1]), (used[3], free[2]), (w.nb, free[3]), (used[1], -1)]
    for s, d in pairs[:3]:
        want[d] = w.cache[s]
    pa.pa_latent_block_copy(w.cache, torch.tensor(pairs, dtype=torch.int64, device=DEV))
    assert same_bits(w.cache, want)


# ------------------------------------------------------------------ absorbed attention

def absorbed(w, heads, news, seed, qscale=1.0, max_len=None, query_start=True, query=None, stream=None):
    """Run the call over Paged w; news[i] new tokens of sequence i (None: decode)."""
    dt = R.TYPES[w.kv]
    n = len(w.lens) if news is None else sum(news)
    if query is None:
        g = torch.Generator().manual_seed(seed)
        query = (torch.randn(n, heads, 576, generator=g) * qscale).to(dt).to(DEV)
    out = torch.full((n, heads, 512), math.inf, dtype=dt, device=DEV)
    mx = max(w.lens + [0]) if max_len is None else max_len
    ws = torch.full((pa.pa_latent_attention_workspace_size(len(w.lens), n, heads, mx),), 255, dtype=torch.uint8,
                    device=DEV)
    qs = None
    if news is not None:
        qs = i32([sum(news[:i]) for i in range(len(news) + 1)])
    pa.pa_latent_attention(out, query, w.cache, w.tables, w.lens_t, SCALE, mx, ws, query_start=qs, stream=stream)
    torch.cuda.synchronize()
    assert pa.pa_workspace_status(ws) == pa.PA_OK
    return query, out


def compare_absorbed(w, query, out, news):
    at = 0
    for i, L in enumerate(w.lens):
        c = w.rows(i)
        for j in range(1 if news is None else news[i]):
            vis = L if news is None else L - news[i] + j + 1
            if vis == 0:
                assert (out[at] == 0).all()
            else:
                o, tol = R.attend(query[at].double(), c[:vis], c[:vis, :512], SCALE, R.TYPES[w.kv])
                R.check(out[at], o, tol, f"sequence {i} of {L}, new token {j}")
            at += 1


@kvs
@pytest.mark.parametrize("heads", [1, 3, 16, 17, 64, 65, 128])
def test_absorbed_decode(kv, heads):
    lens = [1, 2, 63, 64, 65, 127, 129, 300, 0, 1000]
    w = R.Paged(lens, 16, kv, heads, DEV)
    q, out = absorbed(w, heads, None, 1)
    compare_absorbed(w, q, out, None)
    assert same_bits(out, absorbed(w, heads, None, 1)[1])


@kvs
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
def test_absorbed_block_sizes_and_long_contexts(kv, bs):
    lens = [4097, 31, 9000]
    w = R.Paged(lens, bs, kv, bs, DEV)
    q, out = absorbed(w, 16, None, 2)
    compare_absorbed(w, q, out, None)


@kvs
@pytest.mark.parametrize("heads,news", [(16, [4, 1, 3, 4, 0, 2]), (5, [13, 2, 1, 0, 7, 3]), (128, [2, 1, 3, 1, 1, 2]),
                                        (40, [3, 5, 2, 1, 1, 9]), (1, [130, 3, 1, 65, 2, 64])])
def test_absorbed_several_new_tokens(kv, heads, news):
    lens = [max(a, b) for a, b in zip([4, 700, 64, 66, 30, 129], news)]
    w = R.Paged(lens, 16, kv, heads + 1, DEV)
    q, out = absorbed(w, heads, news, 3)
    compare_absorbed(w, q, out, news)
    assert same_bits(out, absorbed(w, heads, news, 3)[1])


@kvs
def test_absorbed_many_sequences(kv):
    lens = [(37 * i) % 500 for i in range(700)]
    w = R.Paged(lens, 32, kv, 77, DEV)
    q, out = absorbed(w, 8, None, 4)
    compare_absorbed(w, q, out, None)


@kvs
def test_absorbed_with_large_scores(kv):
    # scores far apart, of either sign: maxima that jump late, and rows whose
    # first tiles are all far below them
    w = R.Paged([2000, 700, 129], 16, kv, 21, DEV, scale=4.0)
    q, out = absorbed(w, 16, None, 5, qscale=4.0)
    compare_absorbed(w, q, out, None)


@kvs
def test_absorbed_bad_rows(kv):
    lens = [100, 100, 100, 100, 64]
    w = R.Paged(lens, 16, kv, 31, DEV)
    q, ok = absorbed(w, 16, None, 6)
    tables, lens_t = w.tables.clone(), w.lens_t.clone()
    w.tables[1, 3] = w.nb
    w.tables[2, 6] = -7
    w.lens_t[3] = 101                                        # past max_context_len
    _, out = absorbed(w, 16, None, 6, query=q)
    for i in range(5):
        if i in (1, 2, 3):
            assert torch.isnan(out[i]).all(), i
        else:
            assert same_bits(out[i], ok[i]), i
    w.lens_t[3] = -1
    assert torch.isnan(absorbed(w, 16, None, 6, query=q)[1][3]).all()
    w.lens_t[3] = 1000
    assert torch.isnan(absorbed(w, 16, None, 6, query=q, max_len=5000)[1][3]).all()    # past the table
    w.tables, w.lens_t = tables, lens_t


@kvs
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=["nan", "inf", "ninf"])
def test_absorbed_later_new_tokens_do_not_leak(kv, bad):
    # a new token's row that is not finite: earlier new tokens do not see it, and
    # their rows are as if it were not there; itself and later ones are not finite
    heads, news, lens = 16, [6, 3, 9], [200, 64, 70]
    w = R.Paged(lens, 16, kv, 61, DEV)
    q, want = absorbed(w, heads, news, 8)
    flat = w.cache.view(w.nb * w.bs, -1)
    for i, j in ((0, 3), (1, 1), (2, 5)):
        slot = int(w.seq_slots[i][lens[i] - news[i] + j])
        if kv == pa.PA_KV_FP8_E4M3:
            flat[slot, 40] = 0x7f if math.isnan(bad) else flat[slot, 40]
            if not math.isnan(bad):
                flat[slot, 512 + 128:512 + 132].view(torch.float32)[0] = bad
        else:
            flat[slot, 40] = bad
    _, out = absorbed(w, heads, news, 8, query=q)
    at = 0
    for n, first in zip(news, (3, 1, 5)):
        assert same_bits(out[at:at + first], want[at:at + first])
        if not math.isinf(bad):
            assert torch.isnan(out[at + first:at + n]).all()
        else:
            # a score of +inf makes the row NaN; one of -inf takes the token out of
            # it, but for the infinite elements themselves, where the definition
            # has 0 * inf
            rows = out[at + first:at + n].float()
            rows = torch.cat([rows[..., :40], rows[..., 41:128], rows[..., 256:]], -1)
            assert (torch.isnan(rows).all(-1) | torch.isfinite(rows).all(-1)).all()
            assert torch.isnan(rows).any()
        at += n


@kvs
@pytest.mark.parametrize("heads", [16, 128])
def test_absorbed_seen_infinities_reach_the_row(kv, heads):
    # an infinite latent element that a row sees makes the row not finite whatever
    # the sign of its score: 0 * inf in the definition where the score is -inf
    news, lens = [5, 2, 1], [150, 130, 90]
    w = R.Paged(lens, 32, kv, 67, DEV)
    q, want = absorbed(w, heads, news, 12)
    q = q.abs()
    q, want = absorbed(w, heads, news, 12, query=q)
    flat = w.cache.view(w.nb * w.bs, -1)
    for i, j in ((0, 2), (1, 0), (2, 0)):
        slot = int(w.seq_slots[i][lens[i] - news[i] + j])
        if kv == pa.PA_KV_FP8_E4M3:
            flat[slot, 40] = 0xb8                            # -1 times an infinite scale
            flat[slot, 512 + 128:512 + 132].view(torch.float32)[0] = math.inf
        else:
            flat[slot, 40] = -math.inf
    _, out = absorbed(w, heads, news, 12, query=q)
    at = 0
    for n, first in zip(news, (2, 0, 0)):
        assert same_bits(out[at:at + first], want[at:at + first])
        rows = out[at + first:at + n].float()
        assert not torch.isfinite(rows[..., 40]).any()
        at += n


def test_absorbed_longest_contexts():
    # 5,000,001 positions of which a table names 40 blocks again and again: the
    # same as over those blocks' rows weighted by how often they are seen
    bs, nb, n = 64, 40, 5_000_001
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(nb * bs, 576, generator=g).bfloat16()
    q = torch.randn(1, 16, 576, generator=g).bfloat16()
    entries = torch.randint(nb, (-(-n // bs),), generator=g)
    seen = torch.zeros(nb * bs, dtype=torch.float64)
    for k in range(bs):   # the last block is seen up to its remainder
        hit = entries if k < (n - 1) % bs + 1 else entries[:-1]
        seen.view(nb, bs)[:, k] = torch.bincount(hit, minlength=nb).double()
    s = (q[0].double() @ rows.double().T) * SCALE + torch.log(seen)
    want = torch.softmax(s, -1) @ rows[:, :512].double()
    ws = torch.empty(pa.pa_latent_attention_workspace_size(1, 1, 16, n), dtype=torch.uint8, device=DEV)
    out = torch.zeros(1, 16, 512, dtype=torch.bfloat16, device=DEV)
    pa.pa_latent_attention(out, q.to(DEV), rows.view(nb, bs, 576).to(DEV), entries.int()[None].to(DEV), i32([n]), SCALE,
                           2 ** 31 - 1, ws)
    # a probability is rounded by at most 2^-8 of itself and the output by 2^-8 of
    # it; a score's 576 additions (in 32 bits, truncated at worst) lose at most
    # 576 * 2^-23 of the sum of magnitudes, which the softmax doubles; a range of
    # 33,000 positions is 516 tiles of 64 additions to O and to l, a range's piece
    # one of 160
    score = 576 * 2 ** -23 * SCALE * float((q[0].double().abs() @ rows.double().abs().T).max())
    mass = torch.softmax(s, -1) @ rows[:, :512].double().abs()
    bound = (2 ** -8 + 2 * score + 2 * (516 * 64 + 160) * 2 ** -23) * mass + 2 ** -8 * want.abs()
    assert ((out[0].cpu().double() - want).abs() <= bound).all()


def test_absorbed_bad_query_start():
    w = R.Paged([50, 60], 16, pa.PA_KV_BF16, 41, DEV)
    q = torch.randn(6, 16, 576, device=DEV).bfloat16()
    ws = torch.empty(pa.pa_latent_attention_workspace_size(2, 6, 16, 60), dtype=torch.uint8, device=DEV)
    for start in ([0, 4, 3], [1, 4, 6], [0, 7, 6], [0, 3, 5], [0, -1, 6], [0, 3, 7]):
        out = torch.zeros(6, 16, 512, dtype=torch.bfloat16, device=DEV)
        pa.pa_latent_attention(out, q, w.cache, w.tables, w.lens_t, SCALE, 60, ws, query_start=i32(start))
        assert torch.isnan(out).all(), start
    # more new tokens than positions: that sequence only
    out = torch.zeros(6, 16, 512, dtype=torch.bfloat16, device=DEV)
    w.lens_t[0] = 3
    pa.pa_latent_attention(out, q, w.cache, w.tables, w.lens_t, SCALE, 60, ws, query_start=i32([0, 4, 6]))
    assert torch.isnan(out[:4]).all() and torch.isfinite(out[4:]).all()


@kvs
def test_absorbed_captured_and_on_another_stream(kv):
    w = R.Paged([300, 1, 800], 16, kv, 51, DEV)
    q, want = absorbed(w, 16, None, 7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert same_bits(absorbed(w, 16, None, 7, query=q, stream=side)[1], want)
    out = torch.zeros_like(want)
    ws = torch.empty(pa.pa_latent_attention_workspace_size(3, 3, 16, 800), dtype=torch.uint8, device=DEV)
    call = lambda: pa.pa_latent_attention(out, q, w.cache, w.tables, w.lens_t, SCALE, 800, ws)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(out, want)
    w.lens_t.copy_(i32([17, 0, 431]))                        # a replay follows the lengths in the buffers
    w.lens, w.seq_slots = [17, 0, 431], [s[:n] for s, n in zip(w.seq_slots, (17, 0, 431))]
    graph.replay()
    torch.cuda.synchronize()
    compare_absorbed(w, q, out, None)


# ------------------------------------------------------------------ expanded attention

def expanded(dt, news, pasts, heads, seed, poison=True, qscale=1.0):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(news, pasts)]
    nq, nk = sum(news), sum(lens)
    q = (torch.randn(nq, heads, 192, generator=g) * qscale).to(dt).to(DEV)
    up = torch.randn(nk + 9, heads, 264, generator=g).to(dt)     # 8 elements of another operand between heads
    rope = torch.randn(nk + 9, 576, generator=g).to(dt)
    if poison:
        up[nk:], rope[nk:] = math.nan, math.nan
    up, rope = up.to(DEV), rope.to(DEV)
    k, v, r = up[:nk, :, :128], up[:nk, :, 128:256], rope[:nk, 512:]
    out = torch.full((nq, heads, 128), math.inf, dtype=dt, device=DEV)
    qs = i32([sum(news[:i]) for i in range(len(news) + 1)])
    ks = i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    ws = torch.full((pa.pa_latent_attention_expanded_workspace_size(len(news), nq, heads),), 255, dtype=torch.uint8,
                    device=DEV)
    pa.pa_latent_attention_expanded(out, q, k, r, v, qs, ks, SCALE, ws)
    torch.cuda.synchronize()
    assert pa.pa_workspace_status(ws) == pa.PA_OK
    return q, k, r, v, out, (qs, ks, ws)


def compare_expanded(q, k, r, v, out, news, pasts):
    q0 = k0 = 0
    for n, past in zip(news, pasts):
        L = n + past
        for h in range(q.shape[1]):
            key = torch.cat([k[k0:k0 + L, h], r[k0:k0 + L]], 1).double()
            val = v[k0:k0 + L, h].double()
            # rows with the same tolerance formula, each over its own positions
            for j in sorted({0, 1, n // 2, n - 2, n - 1} & set(range(n))) if n > 40 else range(n):
                vis = past + j + 1
                o, tol = R.attend(q[q0 + j, h:h + 1].double(), key[:vis], val[:vis], SCALE, q.dtype)
                R.check(out[q0 + j, h:h + 1], o, tol, f"{n} new after {past}, token {j}, head {h}")
        q0, k0 = q0 + n, k0 + L


types = pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])


@types
@pytest.mark.parametrize("heads,news,pasts", [
    (1, [1], [0]), (2, [1, 5], [0, 70]), (3, [127, 1, 0, 129], [0, 500, 0, 3]), (4, [256, 255, 257], [0, 1, 127]),
    (2, [600, 33], [0, 1000]), (5, [384, 2], [129, 4000]), (1, [128, 64, 300], [128, 64, 212])])
def test_expanded(dt, heads, news, pasts):
    q, k, r, v, out, _ = expanded(dt, news, pasts, heads, 100 + heads + len(news))
    compare_expanded(q, k, r, v, out, news, pasts)
    assert same_bits(out, expanded(dt, news, pasts, heads, 100 + heads + len(news))[4])


@types
def test_expanded_with_large_scores(dt):
    news, pasts = [200, 70], [500, 0]
    q, k, r, v, out, _ = expanded(dt, news, pasts, 2, 7, qscale=16.0)
    compare_expanded(q, k, r, v, out, news, pasts)


@types
def test_expanded_neighbours_do_not_leak(dt):
    # a sequence whose rows are NaN and infinite lies in the same tiles as its
    # neighbours' last keys; their rows are as if it were not there
    news, pasts = [70, 40, 90], [30, 3, 21]
    q, k, r, v, out, (qs, ks, ws) = expanded(dt, news, pasts, 2, 17)
    a, b = 100, 143
    for t, bad in ((k, math.nan), (v, math.inf), (r, math.nan)):
        t[a:b] = bad
    got = torch.zeros_like(out)
    pa.pa_latent_attention_expanded(got, q, k, r, v, qs, ks, SCALE, ws)
    assert same_bits(got[:70], out[:70]) and same_bits(got[110:], out[110:])
    assert torch.isnan(got[70:110]).all()


@types
@pytest.mark.parametrize("bad", [math.nan, math.inf], ids=["nan", "inf"])
def test_expanded_later_new_tokens_do_not_leak(dt, bad):
    # values, keys and rotary keys of new tokens that are not finite: rows of
    # earlier new tokens are as if they were finite, later ones are not finite
    news, pasts = [300, 140, 20], [100, 0, 256]
    q, k, r, v, out, (qs, ks, ws) = expanded(dt, news, pasts, 2, 29)
    # (sequence, new token, tensor, head): the same token may be hit twice
    hits = [(0, 290, v, 0), (0, 130, v, 1), (0, 131, v, 1), (1, 60, k, 0), (1, 139, v, 0), (2, 7, r, None)]
    k0, q0 = [0, 400, 540], [0, 300, 440]
    for i, j, t, h in hits:
        row = k0[i] + pasts[i] + j
        if h is None:
            t[row, 5] = bad
        else:
            t[row, h, 77] = bad
    got = torch.zeros_like(out)
    pa.pa_latent_attention_expanded(got, q, k, r, v, qs, ks, SCALE, ws)
    for i in range(3):
        for h in range(2):
            first = min([j for a, j, t, b in hits if a == i and (b is None or b == h)] + [news[i]])
            a = q0[i]
            assert same_bits(got[a:a + first, h], out[a:a + first, h]), (i, h)
            last = got[a + first:a + news[i], h].float()
            values = all(t is v for b, j, t, c in hits if b == i and (c is None or c == h))
            if values:   # that element at least
                assert not torch.isfinite(last[:, 77]).any(), (i, h)
            elif math.isnan(bad):
                assert torch.isnan(last).all(), (i, h)
            else:
                # an infinite key: +inf makes a row NaN, -inf takes the token out of it
                assert (torch.isnan(last).all(-1) | torch.isfinite(last).all(-1)).all(), (i, h)


def test_expanded_bad_starts():
    dt = torch.bfloat16
    news, pasts = [5, 6], [4, 2]
    q, k, r, v, out, (qs, ks, ws) = expanded(dt, news, pasts, 2, 19)
    for a, b in (([0, 12, 11], ks), ([1, 5, 11], ks), ([0, 5, 10], ks), (qs, [0, 18, 17]), (qs, [0, 9, 16]),
                 (qs, [2, 9, 17]), ([0, 5, 12], ks), (qs, [0, 9, 18])):
        got = torch.zeros_like(out)
        a, b = (x if isinstance(x, torch.Tensor) else i32(x) for x in (a, b))
        pa.pa_latent_attention_expanded(got, q, k, r, v, a, b, SCALE, ws)
        assert torch.isnan(got).all()
    got = torch.zeros_like(out)                              # five new tokens of three: that sequence only
    pa.pa_latent_attention_expanded(got, q, k, r, v, qs, i32([0, 3, 17]), SCALE, ws)
    assert torch.isnan(got[:5]).all() and torch.isfinite(got[5:]).all()


def test_expanded_captured():
    dt = torch.float16
    news, pasts = [300, 20], [40, 0]
    q, k, r, v, want, (qs, ks, ws) = expanded(dt, news, pasts, 3, 23)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_latent_attention_expanded(out, q, k, r, v, qs, ks, SCALE, ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want)


# ------------------------------------------------------------------ together

@kvs
def test_a_serving_run(kv):
    """Two prompts enter the cache; one is extended in a second chunk whose
    prefix is read back and expanded; then speculative steps run in the absorbed
    form, and verification decides what stays.  The absorbed and the expanded
    form are the same attention, so each step's rows agree with a 64-bit
    attention over what the cache holds."""
    dt, H, bs = R.TYPES[kv], 4, 16
    g = torch.Generator(device=DEV).manual_seed(5 + kv)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    wuk, wuv = (rnd(H, 512, 128) / math.sqrt(512.0)).to(dt), (rnd(H, 512, 128) / math.sqrt(512.0)).to(dt)
    al = pa.Allocator(40, bs)
    ids = [0, 1]
    for s in ids:
        al.add_seq(s)
    width = R.ROW8 if kv == pa.PA_KV_FP8_E4M3 else 576
    cache = torch.zeros(40, bs, width, dtype=torch.uint8 if kv == pa.PA_KV_FP8_E4M3 else dt, device=DEV)

    def put(counts):
        rows = rnd(sum(counts), 576).to(dt)
        slots, pairs = al.append(ids, counts)
        assert len(pairs) == 0
        pa.pa_latent_write(rows[:, :512], rows[:, 512:], torch.from_numpy(slots).to(DEV), cache)

    def tables():
        t, lens = al.block_tables(ids, 20)
        return torch.from_numpy(t).to(DEV), torch.from_numpy(lens).to(DEV), lens.tolist()

    for counts in ([100, 33], [70, 1]):                      # prompts, then a second chunk of the first
        put(counts)
        tab, lens_t, lens = tables()
        ks, qs = i32([0, lens[0], sum(lens)]), i32([0, counts[0], sum(counts)])
        rows = torch.empty(sum(lens), 576, dtype=dt, device=DEV)
        pa.pa_latent_read(rows, cache, tab, ks)
        k = torch.einsum("nc,hcd->nhd", rows[:, :512].float(), wuk.float()).to(dt)
        v = torch.einsum("nc,hcd->nhd", rows[:, :512].float(), wuv.float()).to(dt)
        q = rnd(sum(counts), H, 192).to(dt)
        out = torch.empty(sum(counts), H, 128, dtype=dt, device=DEV)
        ws = torch.empty(pa.pa_latent_attention_expanded_workspace_size(2, sum(counts), H), dtype=torch.uint8, device=DEV)
        pa.pa_latent_attention_expanded(out, q, k, rows[:, 512:], v, qs, ks, SCALE, ws)
        compare_expanded(q, k, rows[:, 512:], v, out, counts, [a - b for a, b in zip(lens, counts)])

    put([4, 3])                                              # the last known token and its drafts
    tab, lens_t, lens = tables()
    qn, qr = rnd(7, H, 128), rnd(7, H, 64)
    q = torch.cat([torch.einsum("nhd,hcd->nhc", qn, wuk.float()), qr], 2).to(dt)
    out = torch.empty(7, H, 512, dtype=dt, device=DEV)
    ws = torch.empty(pa.pa_latent_attention_workspace_size(2, 7, H, max(lens)), dtype=torch.uint8, device=DEV)
    pa.pa_latent_attention(out, q, cache, tab, lens_t, SCALE, max(lens), ws, query_start=i32([0, 4, 7]))
    flat = R.rows64(cache)
    at = 0
    logits = []
    for i, n in enumerate((4, 3)):
        t = torch.arange(lens[i], device=DEV)
        c = flat[tab[i].long()[t // bs] * bs + t % bs]
        for j in range(n):
            vis = lens[i] - n + j + 1
            o, tol = R.attend(q[at].double(), c[:vis], c[:vis, :512], SCALE, dt)
            R.check(out[at], o, tol, f"speculative token {j} of sequence {i}")
            logits.append(torch.einsum("hc,hcd->hd", out[at].float(), wuv.float()).reshape(-1)[:50])
            at += 1
    target = torch.softmax(torch.stack(logits) * 3, 1)       # rows of both sequences: drafts + 1 each
    draft = torch.softmax(torch.stack(logits)[[0, 1, 2, 4, 5]] * 3 + rnd(5, 50), 1)
    drafts = draft.argmax(1).int()
    u, pick = torch.rand(5, generator=g, device=DEV), torch.rand(2, generator=g, device=DEV)
    acc, tok = torch.empty(2, dtype=torch.int32, device=DEV), torch.empty(2, 4, dtype=torch.int32, device=DEV)
    pa.pa_verify_drafts(acc, tok, target, draft, drafts, i32([0, 3, 5]), u, pick)
    a, b = R.verify(target.double().cpu().numpy(), draft.double().cpu().numpy(), drafts.tolist(), [0, 3, 5],
                    u.double().tolist(), pick.double().tolist(), 3)
    assert acc.tolist() == a.tolist() and tok.tolist() == b.tolist()


# ------------------------------------------------------------------ calls behind one another

@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_one_another(captured):
    # calls of three kinds queued without a pause, sharing a workspace, each on
    # inputs that the operation before it has just written: as when run alone
    dt = torch.bfloat16
    heads, news = 16, [3, 1, 2]
    w = R.Paged([700, 90, 333], 16, pa.PA_KV_BF16, 71, DEV)
    g = torch.Generator().manual_seed(4)
    nq = sum(news)
    queries = [torch.randn(nq, heads, 576, generator=g).to(dt).to(DEV) for _ in range(4)]
    starts = i32([0, 3, 4, 6])
    alone = [absorbed(w, heads, news, 0, query=q)[1] for q in queries]
    eq, ek, er, ev, ewant, (eqs, eks, _) = expanded(dt, [200, 40], [60, 300], 2, 13)
    ws = torch.full((max(pa.pa_latent_attention_workspace_size(3, nq, heads, 700),
                         pa.pa_latent_attention_expanded_workspace_size(2, 240, 2)),), 255, dtype=torch.uint8, device=DEV)
    query, outs = torch.empty_like(queries[0]), [torch.empty_like(alone[0]) for _ in queries]
    eouts = [torch.empty_like(ewant) for _ in queries]
    probs = torch.rand(7, 1000, generator=g).to(DEV)
    tokens = [torch.empty(2, 4, dtype=torch.int32, device=DEV) for _ in queries]
    kept = [torch.empty(2, dtype=torch.int32, device=DEV) for _ in queries]
    drafts, dstart = torch.randint(1000, (5,), generator=g).int().to(DEV), i32([0, 3, 5])
    u, su = torch.rand(5, generator=g).to(DEV), torch.rand(2, generator=g).to(DEV)

    def run():
        for i, q in enumerate(queries):
            outs[i].zero_()
            query.copy_(q)
            pa.pa_latent_attention(outs[i], query, w.cache, w.tables, w.lens_t, SCALE, 700, ws, query_start=starts)
            eouts[i].zero_()
            pa.pa_latent_attention_expanded(eouts[i], eq, ek, er, ev, eqs, eks, SCALE, ws)
            pa.pa_verify_drafts(kept[i], tokens[i], probs, None, drafts, dstart, u, su)
            pa.pa_verify_drafts(kept[i], tokens[i], probs, None, drafts, dstart, u, su)

    def check():
        torch.cuda.synchronize()
        for i in range(len(queries)):
            assert same_bits(outs[i], alone[i]) and same_bits(eouts[i], ewant)
            assert torch.equal(tokens[i], tokens[0]) and torch.equal(kept[i], kept[0])
            assert (kept[i] >= 0).all()

    if not captured:
        for _ in range(20):
            run()
        check()
        return
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        other = torch.cuda.Stream()
        other.wait_stream(side)
        with torch.cuda.stream(other):   # a branch that joins right before a call
            junk = torch.ones(1 << 20, device=DEV) * 2
        side.wait_stream(other)
        pa.pa_latent_attention(outs[0], queries[0], w.cache, w.tables, w.lens_t, SCALE, 700, ws, query_start=starts)
        run()
    for _ in range(3):
        for t in outs + eouts:
            t.fill_(math.nan)
        graph.replay()
        check()
    del junk
