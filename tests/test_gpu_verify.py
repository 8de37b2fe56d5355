"""pa_verify_drafts against the definition in 64 bits: counts and tokens have to
be equal.  The inputs keep every decision far from its border compared with the
kernel's rounding (twice a float's precision): random numbers fall within 1e-12
of one with a probability below 1e-6 over all the cases here."""
import math

import numpy as np
import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def run(target, draft, drafts, start, u, pick, most, stream=None):
    b = len(start) - 1
    acc = torch.full((b,), -9, dtype=torch.int32, device=DEV)
    tok = torch.full((b, most + 1), -9, dtype=torch.int32, device=DEV)
    t = lambda x, d: torch.as_tensor(np.asarray(x)).to(d).to(DEV)  # noqa: E731
    pa.pa_verify_drafts(acc, tok, target, draft, t(drafts, torch.int32), t(start, torch.int32), t(u, torch.float32),
                        t(pick, torch.float32), stream=stream)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), tok.cpu().numpy()


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def case(kind, counts, vocab, seed, noise=0.8, width=None, greedy=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    nd, b = sum(counts), len(counts)
    width = width or vocab
    start = [0] + np.cumsum(counts).tolist()
    logits = 2 * torch.randn(nd + b, width, generator=g, device=DEV)
    rows = [start[i] + i + j for i, c in enumerate(counts) for j in range(c)]
    target = torch.softmax(logits[:, :vocab], 1)
    draft = torch.softmax(logits[rows][:, :vocab] + noise * torch.randn(nd, vocab, generator=g, device=DEV), 1)
    drafts = draft.argmax(1) if greedy else torch.multinomial(draft, 1, generator=g).view(-1) if nd else draft[:, 0]
    t, q = (torch.full((x.shape[0], width), math.nan, dtype=TYPES[kind], device=DEV) for x in (target, draft))
    t[:, :vocab], q[:, :vocab] = target.to(TYPES[kind]), draft.to(TYPES[kind])
    u = rng.random(nd).astype(np.float32)
    pick = rng.random(b).astype(np.float32)
    return t[:, :vocab], q[:, :vocab], drafts.int().tolist(), start, u, pick


def compare(args, most, draft=True):
    t, q, d, start, u, pick = args
    q = q if draft else None
    acc, tok = run(t, q, d, start, u, pick, most)
    a, b = R.verify(f64(t), f64(q), d, start, u.astype(np.float64), pick.astype(np.float64), most)
    assert acc.tolist() == a.tolist()
    assert tok.tolist() == b.tolist()
    return a


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("vocab,width", [(1, 1), (2, 2), (5, 8), (127, 127), (128, 128), (129, 132), (1000, 1000),
                                         (32003, 32003), (65537, 65544), (131072, 131072)])
def test_against_the_definition(kind, vocab, width):
    counts = [3, 0, 5, 1, 4, 2, 5, 5]
    compare(case(kind, counts, vocab, vocab, width=width), 5)


@pytest.mark.parametrize("kind", list(TYPES))
def test_without_draft_rows(kind):
    # drafts of probability one: a failed draft is left out of the draw
    counts = [4] * 16
    a = compare(case(kind, counts, 777, 5, greedy=True), 4, draft=False)
    assert a.min() < 4


def test_all_counts_of_standing_drafts():
    counts = [7] * 200
    a = compare(case("f32", counts, 211, 6, noise=0.5), 7)
    assert set(a.tolist()) == set(range(8))


def test_more_drafts_than_a_warp():
    t, q, d, start, u, pick = case("f32", [70, 40, 33], 97, 8, noise=0.0)
    u[:] = 0.5                                               # p = q: all stand, until numbers say otherwise
    u[64], u[70 + 32] = 2.0, 2.0
    acc, tok = run(t, q, d, start, u, pick, 70)
    a, b = R.verify(f64(t), f64(q), d, start, u.astype(np.float64), pick.astype(np.float64), 70)
    assert a.tolist() == [64, 32, 33] and acc.tolist() == a.tolist() and tok.tolist() == b.tolist()


def one(p, q, d, u, pick, most=None):
    t, dr = torch.tensor(p, dtype=torch.float32, device=DEV), None
    if q is not None:
        dr = torch.tensor(q, dtype=torch.float32, device=DEV).view(-1, t.shape[1])
    acc, tok = run(t, dr, d, [0, len(d)], u, [pick], len(d) if most is None else most)
    return int(acc[0]), tok[0].tolist()


def test_borders():
    # u q < p is strict and exact
    p = [[0.25, 0.75], [0.5, 0.5]]
    assert one(p, [[0.5, 0.5]], [0], [0.5], 0.0) == (0, [1, -1])          # 0.25 < 0.25 fails; left: 0.25 at 1
    below = float(np.nextafter(np.float32(0.5), np.float32(0)))
    assert one(p, [[0.5, 0.5]], [0], [below], 0.0) == (1, [0, 0])
    # the draw: the smallest v whose running sum passes u * total
    p = [[0.0, 0.25, 0.0, 0.25, 0.5]]
    for u, want in ((0.0, 1), (below / 2, 1), (0.25, 3), (0.5, 4), (1 - 2.0 ** -24, 4)):
        assert one(p, None, [], [], u) == (0, [want]), u
    # a token the draft did not think of, and one the target excludes
    assert one([[0.5, 0.5], [1.0, 0.0]], [[0.0, 1.0]], [0], [0.9], 0.3) == (1, [0, 0])
    assert one([[0.0, 1.0], [1.0, 0.0]], [[1.0, 0.0]], [0], [0.0], 0.3) == (0, [1, -1])


def test_no_weight_left():
    nan, inf = math.nan, math.inf
    # the draft covers the target everywhere: the token is drawn from the target
    assert one([[0.25, 0.25, 0.0], [1, 0, 0]], [[0.5, 0.25, 0.25]], [0], [0.9], 0.6) == (0, [1, -1])
    # no weight at all, infinite weights
    assert one([[0.0, 0.0]], None, [], [], 0.5) == (0, [-1])
    assert one([[0.0, 0.0], [1.0, 0.0]], [[0.5, 0.5]], [1], [0.5], 0.5) == (0, [-1, -1])
    assert one([[inf, 0.5]], None, [], [], 0.5) == (0, [-1])
    # NaN and negative weights count as zero; a NaN number never passes
    assert one([[nan, -3.0, 0.5, nan]], None, [], [], 0.0) == (0, [2])
    assert one([[0.5, 0.5], [1.0, 0.0]], [[0.1, 0.9]], [0], [nan], 0.3) == (0, [0, -1])


def test_bad_sequences():
    t, q, d, start, u, pick = case("f32", [2, 2, 2, 2], 64, 9, noise=0.0)
    u[:] = 0.5
    good, tok = run(t, q, d, start, u, pick, 2)
    assert good.tolist() == [2, 2, 2, 2]
    d2 = list(d)
    d2[2], d2[5] = 64, -1                                    # the first of sequence 1, the second of sequence 2
    acc, tk = run(t, q, d2, start, u, pick, 2)
    assert acc.tolist() == [2, -1, -1, 2] and (tk[1:3] == -1).all() and (tk[[0, 3]] == tok[[0, 3]]).all()
    u2 = u.copy()
    u2[4] = 2.0                                              # a draft before it fails: it is never looked at
    assert run(t, q, d2, start, u2, pick, 2)[0].tolist() == [2, -1, 0, 2]
    for bad in ([0, 2, 1, 6, 8], [0, 2, 4, 6, 7], [1, 2, 4, 6, 8], [0, 2, 4, 9, 8], [0, -1, 4, 6, 8]):
        acc, tk = run(t, q, d, bad, u, pick, 2)
        assert (acc == -1).any() and (tk[acc == -1] == -1).all(), bad
    assert run(t, q, d, [0, 3, 4, 6, 8], u, pick, 2)[0][0] == -1          # three drafts of at most two


@pytest.mark.parametrize("n", [100, 200, 400, 900])
def test_cluster_sizes(n):
    # a sequence's cluster shrinks as the batch grows; rows of odd length, some
    # sequences without drafts, one whose draft covers the target
    counts = [i % 3 for i in range(n)]
    args = list(case("f32", counts, 1501, n))
    t, q, d, start, u, pick = args
    i = next(i for i in range(n) if counts[i] == 2)
    r = start[i]
    q[r] = torch.clamp(t[r + i] * 1.5, min=1e-6)
    u[r] = 0.999
    compare((t, q, d, start, u, pick), 2)


def test_many_sequences_captured():
    counts = [i % 4 for i in range(300)]
    t, q, d, start, u, pick = case("f32", counts, 4099, 10)
    acc, tok = (torch.empty(300, dtype=torch.int32, device=DEV), torch.empty(300, 4, dtype=torch.int32, device=DEV))
    dev = [torch.tensor(x, device=DEV) for x in (np.array(d, dtype=np.int32), np.array(start, dtype=np.int32), u, pick)]
    call = lambda: pa.pa_verify_drafts(acc, tok, t, q, *dev)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    u2 = np.random.default_rng(11).random(len(u)).astype(np.float32)
    dev[2].copy_(torch.tensor(u2))
    graph.replay()
    torch.cuda.synchronize()
    a, b = R.verify(f64(t), f64(q), d, start, u2.astype(np.float64), pick.astype(np.float64), 3)
    assert acc.tolist() == a.tolist() and tok.tolist() == b.tolist()
