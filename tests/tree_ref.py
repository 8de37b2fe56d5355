"""Plain 64-bit forms of the rotation, of attention over trees of drafted tokens,
of their verification and of the move of a path, and seeded inputs for their
tests (tensors on any device)."""
import math

import numpy as np
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa

ROWS = {pa.PA_KV_F16: torch.float16, pa.PA_KV_BF16: torch.bfloat16, pa.PA_KV_FP8_E4M3: torch.float16}
CACHES = {pa.PA_KV_F16: torch.float16, pa.PA_KV_BF16: torch.bfloat16, pa.PA_KV_FP8_E4M3: torch.uint8}


def ids(n, seed, device):
    """A permutation of n blocks."""
    return torch.from_numpy(np.random.default_rng(seed).permutation(n).astype(np.int32)).to(device)


def rotate(x, positions, inv_freq, pair_axis, interleaved):
    """x [n, heads, d] turned in 64 bits; positions [axes, n].  An axis out of range gives NaN."""
    x, pairs = x.double().clone(), inv_freq.shape[0]
    axis = torch.zeros(pairs, dtype=torch.long, device=x.device) if pair_axis is None else pair_axis.long()
    ok = (axis >= 0) & (axis < positions.shape[0])
    angle = positions.double()[torch.where(ok, axis, 0)].T * inv_freq.double()   # [n, pairs]
    angle = torch.where(ok, angle, math.nan)
    c, s = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
    i = torch.arange(pairs, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    u, w = x[..., a], x[..., b]
    x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x


def rotation_bound(x, positions, inv_freq, pair_axis, interleaved, dt):
    """How far a turned element rounded to dt may be from `rotate`'s, by arithmetic.
    The turn's fraction is at most 1/2 and rounded to 24 bits (2^-26 turns, 1e-7 as
    an angle), its 64-bit form off by three roundings of |angle| 2^-53; sine and
    cosine are within two units of their last place (1.2e-7); the two products
    and the sum round three times (3 * 2^-24 = 1.8e-7 of |x| + |y|).  Then half a step of dt."""
    n, pairs = x.shape[0], inv_freq.shape[0]
    axis = torch.zeros(pairs, dtype=torch.long, device=x.device) if pair_axis is None else pair_axis.long()
    angle = (positions.double()[axis.clamp(0, positions.shape[0] - 1)].T * inv_freq.double()).abs()
    size = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    i = torch.arange(pairs, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    both = x[..., a].double().abs() + x[..., b].double().abs()
    err = both * (1e-7 + 1.2e-7 + 1.8e-7 + 2.0 ** -51 * angle.view(n, 1, pairs))
    size[..., a], size[..., b] = err, err
    exact = rotate(x, positions, inv_freq, pair_axis, interleaved).abs()
    least = 2.0 ** -25 if dt == torch.float16 else 0.0    # half a subnormal step
    return size + (exact + size) * R.half_step(dt) + least


def ancestors(parents):
    """[T, T] truth values: what each node of one tree sees of it."""
    T = len(parents)
    sees = np.zeros((T, T), dtype=bool)
    for j in range(T):
        a = j
        while a >= 0:
            sees[j, a] = True
            assert parents[a] < a
            a = parents[a]
    return torch.from_numpy(sees)


def cached(cache, table, n, bs, unit):
    """Rows of a sequence's first n positions [n, kv_heads, d] in 64 bits."""
    pos = torch.arange(n, device=cache.device)
    x = cache[table.long()[pos // bs], :, pos % bs]
    return (R.e4m3_value(x) if x.dtype == torch.uint8 else x.double()) * unit


def tree_attention(q, k, v, sees, scale, dt):
    """(out, bound) of one sequence in 64 bits: q [T, hq, d], k and v [L, hk, d], sees [T, L].

    The bound: a probability is off by its score's error and by its rounding to dt.
    A score's d products are exact and their sum is carried in 24 bits or nearly so
    (2^-20 of the sum of magnitudes), as is its product with the scale; exp2 is good
    to 2^-21.  Relative to a row's sum these weigh |v|, twice because the sum is off
    too.  Probabilities below a subnormal's half step lose at most 2^-25 (fp16) each,
    against a sum of at least the largest one's 1.  Then the output's half step."""
    T, hq, d = q.shape
    hk, half = k.shape[1], R.half_step(dt)
    least = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -133
    outs, bounds = [], []
    for h in range(hq):
        g = h * hk // hq
        s = q[:, h].double() @ k[:, g].T * scale
        s = s.masked_fill(~sees, -math.inf)
        size = (q[:, h].double().abs() @ k[:, g].abs().T * scale).masked_fill(~sees, 0.0).amax(1, keepdim=True)
        p = torch.exp(s - s.amax(1, keepdim=True))
        l = p.sum(1, keepdim=True)
        vh = torch.where(sees.any(0).view(-1, 1), v[:, g], 0.0)
        o, mass = p @ vh / l, p @ vh.abs() / l
        err = mass * (half + 2 * (size * 2.0 ** -20 + 2.0 ** -21) + 2.0 ** -20)
        err = err + sees.sum(1, keepdim=True) * least * vh.abs().amax() / l
        outs.append(o)
        bounds.append(err + (o.abs() + err) * half + least)
    return torch.stack(outs, 1), torch.stack(bounds, 1)


def verify_tree(target, tokens, parents, start, u, depth):
    """(accepted, tokens, path) by the definition; target float64 [nodes, vocab] on the host."""
    b = len(start) - 1
    acc = np.full(b, -1, dtype=np.int32)
    out, path = (np.full((b, depth + 1), -1, dtype=np.int32) for _ in range(2))
    for i in range(b):
        n0, n1 = start[i], start[i + 1]
        node = 0 if n1 > n0 else -1
        while node >= 0:
            acc[i] += 1
            w = np.nan_to_num(target[n0 + node], nan=0.0, posinf=math.inf, neginf=0.0).clip(min=0.0)
            c = np.cumsum(w)
            v = -1
            if 0.0 < c[-1] < math.inf:
                v = int(np.searchsorted(c, u[n0 + node] * c[-1], side="right"))
            out[i, acc[i]], path[i, acc[i]] = v, node
            kids = [j for j in range(node + 1, n1 - n0) if parents[n0 + j] == node and tokens[n0 + j] == v]
            node = kids[0] if kids and v >= 0 and acc[i] < depth else -1
    return acc, out, path


def random_tree(rng, n, kind):
    """Parents of a tree of n nodes, parents first: a chain, a bush (everything below the root), by levels, at random,
    or several roots beside one another."""
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "bush":
        return [-1] + [0] * (n - 1)
    if kind == "levels":
        return [-1] + [(j - 1) // 2 for j in range(1, n)]
    if kind == "roots":
        return [-1 if j % 3 == 0 else j - 1 for j in range(n)]
    return [-1] + [int(rng.integers(0, j)) for j in range(1, n)]


KINDS = ["chain", "bush", "levels", "random", "roots"]
