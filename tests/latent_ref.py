"""Plain 64-bit forms of the latent-cache operators and of draft verification,
and seeded inputs for their tests (tensors on any device)."""
import math

import numpy as np
import torch

import paged_kv_cache_12_gb300 as pa

DC, DR, ROW, ROW8 = pa.PA_LATENT_DIM, pa.PA_LATENT_ROPE_DIM, pa.PA_LATENT_ROW, pa.PA_LATENT_ROW_FP8_BYTES
TYPES = {pa.PA_KV_F16: torch.float16, pa.PA_KV_BF16: torch.bfloat16, pa.PA_KV_FP8_E4M3: torch.bfloat16}
KVS = [pa.PA_KV_F16, pa.PA_KV_BF16, pa.PA_KV_FP8_E4M3]
KV_IDS = ["f16", "bf16", "fp8"]


def half_step(dt):
    return torch.finfo(dt).eps / 2


def e4m3_value(code):
    """Values of E4M3 codes (uint8), from the format's definition; NaN at 0x7f and 0xff."""
    c = code.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m * 2.0 ** -9)
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag)


ALL_CODES = e4m3_value(torch.arange(256, dtype=torch.uint8))


def encode_e4m3(y):
    """The code of the nearest E4M3 value, ties to the even code, saturating; by
    search over the finite magnitudes.  NaN -> 0x7f."""
    mags = ALL_CODES[:127].to(y.device)
    a = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(mags, a.nan_to_num(0.0)).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - mags[lo], mags[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(torch.isnan(y), torch.full_like(code, 127), code)
    return torch.where(torch.signbit(y) & ~torch.isnan(y), code + 128, code).to(torch.uint8)


def quantise(latent):
    """bf16 [n, 512] -> codes [n, 512], float64 scales [n, 4]."""
    x = latent.double().view(-1, 4, 128)
    top = x.abs().nan_to_num(0.0, posinf=float(torch.finfo(torch.bfloat16).max)).amax(2)
    e = torch.full_like(top, -100.0)
    for k in range(-100, 119):   # the smallest exponent that holds the group
        e = torch.where(top > 448.0 * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    return encode_e4m3((x * torch.exp2(-e).unsqueeze(2)).reshape(-1, DC)), torch.exp2(e)


def pack8(latent, rope):
    """Quantised rows as bytes [n, 656]."""
    codes, scales = quantise(latent)
    return torch.cat([codes, rope.contiguous().view(torch.uint8).view(-1, 2 * DR),
                      scales.float().contiguous().view(torch.uint8).view(-1, 16)], 1)


def rows64(cache):
    """float64 rows [slots, 576] of a latent cache."""
    if cache.dtype != torch.uint8:
        return cache.reshape(-1, ROW).double()
    r = cache.reshape(-1, ROW8)
    scales = r[:, DC + 2 * DR:].contiguous().view(torch.float32).double()
    latent = e4m3_value(r[:, :DC]).view(-1, 4, 128) * scales.unsqueeze(2)
    return torch.cat([latent.reshape(-1, DC), r[:, DC:DC + 2 * DR].contiguous().view(torch.bfloat16).double()], 1)


def nan_cache(nb, bs, kv, device):
    """A cache whose every element is NaN (codes 0x7f, NaN rotary elements and scales)."""
    if kv == pa.PA_KV_FP8_E4M3:
        c = torch.full((nb, bs, ROW8), 0x7f, dtype=torch.uint8, device=device)
        c[..., DC + 2 * DR:] = 0xff
        c[..., DC:DC + 2 * DR] = 0xff
        return c
    return torch.full((nb, bs, ROW), math.nan, dtype=TYPES[kv], device=device)


class Paged:
    """Sequences of the given lengths over a shuffled, NaN-poisoned pool: slots
    that hold no token are NaN."""

    def __init__(self, lens, bs, kv, seed, device, spare=3, scale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + spare
        order = rng.permutation(nb)
        self.kv, self.bs, self.lens, self.nb = kv, bs, list(lens), nb
        self.tables_np = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.tables_np[i, :n] = order[at:at + n]
            at += n
        self.cache = nan_cache(nb, bs, kv, "cpu")
        flat = self.cache.view(nb * bs, -1)
        self.seq_slots = []
        for i, n in enumerate(lens):
            t = torch.arange(n)
            slots = torch.from_numpy(self.tables_np[i].astype(np.int64))[t // bs] * bs + t % bs
            self.seq_slots.append(slots)
            x = (torch.randn(n, ROW, generator=g) * scale).to(TYPES[kv])
            if n:
                flat[slots] = pack8(x[:, :DC], x[:, DC:]) if kv == pa.PA_KV_FP8_E4M3 else x
        self.cache = self.cache.to(device)
        self.tables = torch.from_numpy(self.tables_np).to(device)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=device)

    def rows(self, i):
        """float64 rows of sequence i, on the cache's device."""
        return rows64(self.cache.view(self.nb * self.bs, -1)[self.seq_slots[i].to(self.cache.device)])


def attend(q, k, v, scale, dt):
    """softmax(scale q k^T) v in float64 for query rows q [h, dk] over one list
    of positions, and how far a kernel may be from it element by element.

    The kernel's roundings: products are exact in fp32 and a score's sum of dk of
    them is off by at most dk 2^-24 sum|q k| scale =: d, which moves a
    probability by a relative 2 d (numerator and denominator); each probability
    is rounded to the 16-bit type (half a step u); n terms accumulate in fp32
    (n 2^-24); exponentials and merges stay below 2^-20.  All of these scale
    E = sum p |v|.  The result is rounded once more (u |o|).  An fp16
    probability below 2^-14 (relative to one no smaller than the largest / 2^8)
    is off by at most 2^-25 absolutely instead."""
    n = k.shape[0]
    s = q @ k.T * scale
    p = torch.softmax(s, 1)
    o = p @ v
    u = half_step(dt)
    d = (q.abs() @ k.abs().T).amax(1, keepdim=True) * scale * q.shape[1] * 2.0 ** -24
    tol = (u + 2 * d + n * 2.0 ** -24 + 2.0 ** -20) * (p @ v.abs()) + u * o.abs()
    if dt == torch.float16:
        tol = tol + n * 2.0 ** -25 * v.abs().amax(0) + 2.0 ** -25
    return o, tol


def check(got, want, tol, where=""):
    got = got.double()
    assert torch.isfinite(got).all(), where + ": not finite"
    worst = ((got - want).abs() / tol).max().item()
    assert worst <= 1.0, f"{where}: {worst:.2f} times the tolerance"


def verify(target, draft, drafts, start, u, pick, most):
    """(accepted, tokens) from the definition in 64 bits; rows are numpy float64."""
    accepted, tokens = [], []
    for i in range(len(start) - 1):
        a, n, row = 0, start[i + 1] - start[i], []
        while a < n:
            r, d = start[i] + a, drafts[start[i] + a]
            q = 1.0 if draft is None else draft[r][d]
            if not u[r] * q < target[r + i][d]:
                break
            row.append(int(d))
            a += 1
        p = target[start[i] + i + a]
        w = p
        if a < n:
            if draft is None:
                w = p.copy()
                w[drafts[start[i] + a]] = 0.0
            else:
                w = p - draft[start[i] + a]
        w = np.where(w > 0, w, 0.0)
        if a < n and w.sum() == 0:
            w = np.where(p > 0, p, 0.0)
        c = np.cumsum(w)
        if c[-1] > 0 and np.isfinite(c[-1]):
            row.append(int(np.searchsorted(c, pick[i] * c[-1], side="right")))
        else:
            row.append(-1)
        accepted.append(a)
        tokens.append(row + [-1] * (most + 1 - len(row)))
    return np.array(accepted), np.array(tokens)
