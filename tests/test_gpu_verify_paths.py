"""pa_verify_drafts on the paths that depend on the batch: slices longer than
what a warp sums at once, searched in parts, in clusters of four, two and one
CTA.  Counts and tokens have to be equal to the definition's in 64 bits."""
import numpy as np
import pytest
import torch

from test_gpu_verify import case, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(100, 32003), (200, 20011), (400, 9001), (500, 65537)])
def test_long_slices_in_small_clusters(kind, n, vocab):
    # (a GPU of 152 SMs takes clusters of 4 from 77 sequences on, of 2 from 153 and
    # of 1 from 305.)  Heights at both ends of the sum, in the middle, and drafts
    # that cover the target, whose draw is made from the target itself
    counts = [i % 3 if n < 500 else i % 2 for i in range(n)]
    t, q, d, start, u, pick = case(kind, counts, vocab, n + vocab)
    below = 1 - 2.0 ** -24
    pick[0:40:4] = 0.0
    pick[1:40:4] = below
    pick[2:40:4] = np.linspace(0.1, 0.9, 10).astype(np.float32)
    covered = [i for i in range(n) if counts[i] == max(counts)][::7]
    for i in covered:
        r = start[i]
        q[r] = torch.clamp(t[r + i].float() * 1.5, min=1e-6).to(q.dtype)
        u[r] = 0.999
    pick[covered[0]], pick[covered[1]] = 0.0, below
    compare((t, q, d, start, u, pick), max(counts))


@pytest.mark.parametrize("n,vocab", [(200, 37), (4, 32003), (100, 32003), (400, 9001)])
def test_weights_next_to_the_smallest_float(n, vocab):
    # rows need not sum to one: weights of a few times 2^-149 each, where a height
    # u * total rounded to a float's steps passes other sums than it should
    g = np.random.default_rng(n + vocab)
    rows = g.integers(0, 4, size=(n, vocab)).astype(np.float64) * 2.0 ** -149
    target = torch.tensor(rows.astype(np.float32), device="cuda")
    assert (target.double().cpu().numpy() == rows).all()
    pick = g.random(n).astype(np.float32)
    compare((target, target[:0], [], [0] * (n + 1), np.zeros(0, dtype=np.float32), pick), 0)
