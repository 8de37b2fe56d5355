"""The operators of a latent KV cache and of speculative steps, as cases that can be timed and checked.

Every case is one call that a serving program makes:

  write     rows of a step's new tokens (a 512-wide latent and a 64-wide rotary key each) into the paged latent cache,
            as 16-bit rows or quantised to one-byte codes
  read      cached rows of whole sequences back into contiguous 16-bit rows
  absorbed  attention over the latent cache, queries already multiplied into the latent space
  expanded  causal attention over keys and values expanded per head from the latents
  verify    drafted tokens against the target's probabilities, from given random numbers

``run`` computes a case with elementary torch operations in 32 bits or more; with ``own`` set it makes the framework's
calls instead.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DC, DR = 512, 64              # latent and rotary widths of a cached row
ROW8 = DC + 2 * DR + 16       # bytes of a quantised row: codes, bf16 rotary key, four float scales
DN, DV = 128, 128             # expanded per-head widths: key without its rotary part, value
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's rows of 100 sequences into a 16-bit cache: latency
        {"name": "write_step_f16", "op": "write", "cache": "f16", "tokens": 100, "block": 16},
        # prompts of a whole step quantised as they are written
        {"name": "write_prompts_fp8", "op": "write", "cache": "fp8", "tokens": 65536, "block": 32},
        # a cached 12000-token prompt read back before its next chunk is expanded
        {"name": "read_prompt_bf16", "op": "read", "cache": "bf16", "seqs": 1, "lo": 12000, "hi": 12000, "block": 16},
        # a ragged batch of quantised contexts read back
        {"name": "read_ragged_fp8", "op": "read", "cache": "fp8", "seqs": 64, "lo": 64, "hi": 8192, "block": 16},
        # one chat request alone: latency
        {"name": "absorbed_one_bf16", "op": "absorbed", "cache": "bf16", "seqs": 1, "lo": 600, "hi": 600, "heads": 16,
         "new": 1, "block": 16},
        # a full decode batch on one of several tensor-parallel shards
        {"name": "absorbed_batch_bf16", "op": "absorbed", "cache": "bf16", "seqs": 100, "lo": 8192, "hi": 8192,
         "heads": 16, "new": 1, "block": 16},
        # all heads on one GPU, contexts from a question to a book chapter
        {"name": "absorbed_mix_f16", "op": "absorbed", "cache": "f16", "seqs": 96, "lo": 64, "hi": 32768, "heads": 128,
         "new": 1, "block": 32},
        # a speculative step of four new tokens a sequence over a quantised cache
        {"name": "absorbed_spec_fp8", "op": "absorbed", "cache": "fp8", "seqs": 100, "lo": 1024, "hi": 8192,
         "heads": 16, "new": 4, "block": 16},
        # one short prompt from its first token
        {"name": "expanded_prompt_f16", "op": "expanded", "dtype": "f16", "seqs": 1, "new": 600, "past": 0,
         "heads": 16},
        # the last 2048-token chunk of a 12000-token prompt
        {"name": "expanded_chunk_bf16", "op": "expanded", "dtype": "bf16", "seqs": 1, "new": 2048, "past": 9952,
         "heads": 32},
        # a few interactive requests, small odd vocabulary
        {"name": "verify_few_f32", "op": "verify", "probs": "f32", "seqs": 4, "drafts": 4, "vocab": 32003},
        # a full batch of speculative requests, large vocabulary
        {"name": "verify_batch_f32", "op": "verify", "probs": "f32", "seqs": 100, "drafts": 4, "vocab": 131072},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "absorbed", "absorbed", "expanded", "verify"])
    block = rng.choice([8, 16, 32, 64])
    cache = rng.choice(["f16", "bf16", "fp8"])
    if op == "write":
        return {"op": op, "cache": cache, "tokens": _log(rng, 1, 65536), "block": block}
    if op == "read":
        lo = _log(rng, 1, 2000)
        return {"op": op, "cache": cache, "seqs": _log(rng, 1, 48), "lo": lo, "hi": _log(rng, lo, 8192),
                "block": block}
    if op == "absorbed":
        new = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        lo = _log(rng, max(1, new), 8192)
        heads = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 128])
        return {"op": op, "cache": cache, "seqs": _log(rng, 1, 48), "lo": lo, "hi": _log(rng, lo, 16384),
                "heads": heads, "new": min(new, max(1, 256 // heads)), "block": block}
    if op == "expanded":
        new = _log(rng, 1, 2048)
        return {"op": op, "dtype": rng.choice(["f16", "bf16"]), "seqs": _log(rng, 1, 3), "new": new,
                "past": rng.choice([0, _log(rng, 1, 4000)]), "heads": rng.choice([1, 4, 16, 20])}
    return {"op": op, "probs": rng.choice(["f32", "f32", "bf16", "f16"]), "seqs": _log(rng, 1, 64),
            "drafts": rng.choice([1, 2, 3, 4, 7]), "vocab": _log(rng, 500, 131072)}


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spread over their logarithm, in a fixed shuffled order."""
    return [int(round(lo * (hi / lo) ** ((0.5 + i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _lens(case):
    return _spread(case["seqs"], case["lo"], case["hi"])


def _news(case):
    """New tokens of each sequence of a prompt step: the largest first, the others shorter."""
    return [max(1, int(case["new"] * (1.0 - 0.37 * i / max(1, case["seqs"])))) for i in range(case["seqs"])]


def _drafts(case):
    """Drafted tokens of each sequence; some requests bring fewer."""
    return [case["drafts"] if i % 5 != 4 else case["drafts"] - 1 for i in range(case["seqs"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def _quantised(latent):
    """float [n, 512] -> codes (E4M3 values) [n, 512] and scales [n, 4], powers of two: the smallest 2^e (e from -100
    to 119) with max |x| <= 448 * 2^e in each group of 128."""
    x = latent.view(-1, 4, DC // 4)
    f, k = torch.frexp(x.abs().amax(dim=2))
    e = torch.where(f <= 0.875, k - 9, k - 8)
    e = torch.where(f == 0, torch.full_like(e, -100), e).clamp(-100, 119)
    codes = torch.ldexp(x, -e.unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(-1, DC), torch.ldexp(torch.ones_like(f), e)


def _parts(cache):
    """Views of a quantised cache [blocks, block, 656] bytes: codes, rotary keys, scales."""
    return (cache[..., :DC].view(torch.float8_e4m3fn), cache[..., DC:DC + 2 * DR].view(torch.bfloat16),
            cache[..., DC + 2 * DR:].view(torch.float32))


def _pool(case, g, lens):
    """A cache whose every slot holds a row, and the block tables of sequences placed over it at random."""
    bs = case["block"]
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    if case["cache"] == "fp8":
        cache = torch.empty(nb, bs, ROW8, dtype=torch.uint8, device=DEV)
        codes, rope, scales = _parts(cache)
        c, s = _quantised(_randn(g, nb * bs, DC))
        codes.copy_(c.view(nb, bs, DC))
        scales.copy_(s.view(nb, bs, 4))
        rope.copy_(_randn(g, nb, bs, DR))
    else:
        cache = _randn(g, nb, bs, DC + DR).to(DTYPES[case["cache"]])
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = ids[at:at + n]
        at += n
    return cache, tables


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "write":
        n, bs = case["tokens"], case["block"]
        dt = DTYPES.get(case["cache"], torch.bfloat16)
        nb = -(-n // bs) + 5
        # latents and rotary keys as two slices of one projection's rows; every 16th row is padding
        rows = _randn(g, n, DC + DR).to(dt)
        s["latent"], s["rope"] = rows[:, :DC], rows[:, DC:]
        slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n]
        slots[7::16] = -1
        s["slots"] = slots
        if case["cache"] == "fp8":
            s["cache"] = torch.zeros(nb, bs, ROW8, dtype=torch.uint8, device=DEV)
            s["held"] = _parts(s["cache"])
        else:
            s["cache"] = torch.zeros(nb, bs, DC + DR, dtype=dt, device=DEV)
    elif op == "read":
        lens = _lens(case)
        s["cache"], s["tables"] = _pool(case, g, lens)
        s["row_start"] = _i32(_starts(lens))
        s["out"] = torch.empty(sum(lens), DC + DR, dtype=DTYPES.get(case["cache"], torch.bfloat16), device=DEV)
    elif op == "absorbed":
        lens, t, h = _lens(case), case["new"], case["heads"]
        dt = DTYPES.get(case["cache"], torch.bfloat16)
        s["cache"], s["tables"] = _pool(case, g, lens)
        s["lens"], s["max_len"] = _i32(lens), max(lens)
        s["query"] = _randn(g, len(lens) * t, h, DC + DR).to(dt)
        s["query_start"] = None if t == 1 else _i32([i * t for i in range(len(lens) + 1)])
        s["scale"] = 1.0 / math.sqrt(DN + DR)
        s["out"] = torch.empty(len(lens) * t, h, DC, dtype=dt, device=DEV)
    elif op == "expanded":
        news, h, dt = _news(case), case["heads"], DTYPES[case["dtype"]]
        nq, nk = sum(news), sum(news) + case["past"] * len(news)
        s["query"] = _randn(g, nq, h, DN + DR).to(dt)
        up = _randn(g, nk, h, DN + DV).to(dt)                  # one product gives keys and values, head by head
        s["k_nope"], s["value"] = up[..., :DN], up[..., DN:]
        s["k_rope"] = _randn(g, nk, DC + DR).to(dt)[:, DC:]    # the rotary part of the rows that were read back
        s["query_start"], s["kv_start"] = _i32(_starts(news)), _i32(_starts([n + case["past"] for n in news]))
        s["max_new"], s["max_len"] = max(news), max(news) + case["past"]
        s["scale"] = 1.0 / math.sqrt(DN + DR)
        s["out"] = torch.empty(nq, h, DV, dtype=dt, device=DEV)
    else:
        counts, v = _drafts(case), case["vocab"]
        nd, nb = sum(counts), case["seqs"]
        dt = {"f32": torch.float32, **DTYPES}[case["probs"]]
        # the draft model's logits are the target's with noise, so that about two drafts of three pass
        logits = 2.0 * _randn(g, nd + nb, v)
        s["target"] = torch.softmax(logits, dim=1).to(dt)
        rows = torch.tensor([r + i for i, c in enumerate(counts) for r in range(sum(counts[:i]), sum(counts[:i]) + c)],
                            dtype=torch.int64, device=DEV)
        draft = torch.softmax(logits[rows] + 0.8 * _randn(g, nd, v), dim=1)
        pick = torch.rand(nd, 1, generator=g, device=DEV, dtype=torch.float64)
        c = draft.double().cumsum(1)
        s["drafts"] = torch.searchsorted(c, pick * c[:, -1:], right=True).clamp(max=v - 1).view(-1).to(torch.int32)
        s["draft"] = draft.to(dt)
        s["start"] = _i32(_starts(counts))
        s["uniform"] = torch.rand(nd, generator=g, device=DEV, dtype=torch.float32)
        s["pick"] = torch.rand(nb, generator=g, device=DEV, dtype=torch.float32)
        s["accepted"] = torch.empty(nb, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(nb, case["drafts"] + 1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms and the framework's calls

def _float_rows(cache, slots):
    """Cached rows at the given slots as floats [..., 576]."""
    if cache.dtype != torch.uint8:
        return cache.view(-1, DC + DR)[slots].float()
    row = cache.view(-1, ROW8)[slots]
    codes, rope, scales = _parts(row)
    return torch.cat([codes.float() * scales.repeat_interleave(DC // 4, dim=-1), rope.float()], dim=-1)


def _write(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    if s["cache"].dtype == torch.uint8:
        codes, scales = _quantised(s["latent"][keep].float())
        hc, hr, hs = s["held"]
        bs = hc.shape[1]
        hc[at // bs, at % bs] = codes
        hr[at // bs, at % bs] = s["rope"][keep]
        hs[at // bs, at % bs] = scales
        return list(s["held"])
    s["cache"].view(-1, DC + DR)[at] = torch.cat([s["latent"], s["rope"]], dim=1)[keep]
    return s["cache"]


def _read(s):
    n, bs = s["out"].shape[0], s["cache"].shape[1]
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(s["row_start"].long(), row, right=True) - 1
    t = row - s["row_start"].long()[seq]
    slots = s["tables"].long()[seq, t // bs] * bs + t % bs
    return _float_rows(s["cache"], slots).to(s["out"].dtype)


def _absorbed(s):
    b, bs = s["lens"].shape[0], s["cache"].shape[1]
    nq, h, _ = s["query"].shape
    t = nq // b
    pos = torch.arange(s["max_len"], device=DEV)
    lens = s["lens"].long().view(b, 1)
    slots = torch.where(pos < lens, s["tables"].long()[:, pos // bs] * bs + pos % bs, 0)
    kv = _float_rows(s["cache"], slots)
    q = s["query"].float().view(b, t * h, DC + DR)
    score = torch.matmul(q, kv.transpose(1, 2)).view(b, t, h, -1) * s["scale"]
    last = (lens - t + torch.arange(t, device=DEV)).view(b, t, 1, 1)       # the last position each new token sees
    score = score.masked_fill(pos > last, -math.inf)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    return torch.matmul(p.view(b, t * h, -1), kv[..., :DC]).view(nq, h, DC).to(s["query"].dtype)


def _expanded(s):
    nq, h, _ = s["query"].shape
    b = s["query_start"].shape[0] - 1
    q0, k0 = s["query_start"].long(), s["kv_start"].long()
    tq, tk = (q0[1:] - q0[:-1]).view(b, 1), (k0[1:] - k0[:-1]).view(b, 1)
    i, pos = torch.arange(s["max_new"], device=DEV), torch.arange(s["max_len"], device=DEV)
    qi = torch.where(i < tq, q0[:-1].view(b, 1) + i, 0)
    ki = torch.where(pos < tk, k0[:-1].view(b, 1) + pos, 0)
    q = s["query"][qi].float().transpose(1, 2)                             # [b, h, new, 192]
    k, v = s["k_nope"][ki].float().transpose(1, 2), s["value"][ki].float().transpose(1, 2)
    r = s["k_rope"][ki].float().view(b, 1, -1, DR)
    score = (torch.matmul(q[..., :DN], k.transpose(2, 3)) + torch.matmul(q[..., DN:], r.transpose(2, 3))) * s["scale"]
    score = score.masked_fill(pos > (tk - tq + i).view(b, 1, -1, 1), -math.inf)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    out = torch.matmul(p / p.sum(dim=-1, keepdim=True), v).transpose(1, 2)  # [b, new, h, 128]
    row = torch.arange(nq, device=DEV)
    seq = torch.searchsorted(q0, row, right=True) - 1
    return out[seq, row - q0[seq]].to(s["query"].dtype)


def _verify(s):
    nb, most = s["tokens"].shape[0], s["tokens"].shape[1] - 1
    d0 = s["start"].long()
    n = (d0[1:] - d0[:-1]).view(nb, 1)
    j = torch.arange(most, device=DEV)
    seq = torch.arange(nb, device=DEV)
    has = j < n
    at = torch.where(has, d0[:-1].view(nb, 1) + j, 0)
    drafted = s["drafts"].long()[at]
    p = s["target"][at + seq.view(nb, 1), drafted].double()
    q = s["draft"][at, drafted].double()
    passed = (s["uniform"].double()[at] * q < p) & has
    kept = torch.cumprod(passed.long(), dim=1).sum(dim=1)                  # drafts before the first that fails
    target = s["target"][d0[:-1] + seq + kept].double()
    failed = (kept < n.view(nb)).view(nb, 1)
    draft = s["draft"][torch.where(failed.view(nb), d0[:-1] + kept, 0)].double()
    w = torch.clamp(target - torch.where(failed, draft, 0.0), min=0.0)
    c = w.cumsum(dim=1)
    new = torch.searchsorted(c, s["pick"].double().view(nb, 1) * c[:, -1:], right=True).clamp(max=w.shape[1] - 1)
    col = torch.arange(most + 1, device=DEV)
    drafted = torch.cat([drafted, drafted[:, :1]], dim=1)
    kept = kept.view(nb, 1)
    tokens = torch.where(col < kept, drafted, torch.where(col == kept, new, -1))
    return [kept.view(nb).to(torch.int32), tokens.to(torch.int32)]


def _run_own(s):
    import paged_kv_cache_12_gb300 as pa

    op = s["case"]["op"]
    if op == "write":
        pa.pa_latent_write(s["latent"], s["rope"], s["slots"], s["cache"])
        return list(s["held"]) if "held" in s else s["cache"]
    if op == "read":
        pa.pa_latent_read(s["out"], s["cache"], s["tables"], s["row_start"])
        return s["out"]
    if op == "absorbed":
        if "workspace" not in s:
            nq, h, _ = s["query"].shape
            size = pa.pa_latent_attention_workspace_size(s["lens"].shape[0], nq, h, s["max_len"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        pa.pa_latent_attention(s["out"], s["query"], s["cache"], s["tables"], s["lens"], s["scale"], s["max_len"],
                               s["workspace"], query_start=s["query_start"])
        return s["out"]
    if op == "expanded":
        if "workspace" not in s:
            nq, h, _ = s["query"].shape
            size = pa.pa_latent_attention_expanded_workspace_size(s["query_start"].shape[0] - 1, nq, h)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        pa.pa_latent_attention_expanded(s["out"], s["query"], s["k_nope"], s["k_rope"], s["value"], s["query_start"],
                                        s["kv_start"], s["scale"], s["workspace"])
        return s["out"]
    pa.pa_verify_drafts(s["accepted"], s["tokens"], s["target"], s["draft"], s["drafts"], s["start"], s["uniform"],
                        s["pick"])
    return [s["accepted"], s["tokens"]]


def run(state):
    if own:
        return _run_own(state)
    return {"write": _write, "read": _read, "absorbed": _absorbed, "expanded": _expanded,
            "verify": _verify}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    return ROW8 if case["cache"] == "fp8" else 2 * (DC + DR)


def work(case):
    op = case["op"]
    if op == "write":
        n = case["tokens"] - (case["tokens"] + 8) // 16      # rows that are not padding
        return {"bytes": n * (2 * (DC + DR) + _row_bytes(case)) + 8 * case["tokens"], "flops": 0}
    if op == "read":
        n = sum(_lens(case))
        return {"bytes": n * (2 * (DC + DR) + _row_bytes(case)) + 4 * sum(-(-x // case["block"]) for x in _lens(case)),
                "flops": 0}
    if op == "absorbed":
        lens, t, h = _lens(case), case["new"], case["heads"]
        seen = sum(t * x - t * (t - 1) // 2 for x in lens)   # positions seen, over all new tokens
        return {"bytes": sum(lens) * _row_bytes(case) + len(lens) * t * h * 2 * (DC + DR + DC)
                + 4 * sum(-(-x // case["block"]) for x in lens), "flops": 2 * h * seen * (DC + DR + DC)}
    if op == "expanded":
        news, h = _news(case), case["heads"]
        seen = sum(n * case["past"] + n * (n + 1) // 2 for n in news)
        nq, nk = sum(news), sum(news) + case["past"] * len(news)
        return {"bytes": 2 * (nq * h * (DN + DR + DV) + nk * (h * (DN + DV) + DR)),
                "flops": 2 * h * seen * (DN + DR + DV)}
    # one row of the target for each sequence, and the draft's row beside it where a draft failed (about two in
    # three pass); two numbers and a token for each draft
    size = 4 if case["probs"] == "f32" else 2
    rows = sum(2.0 - 0.67 ** n for n in _drafts(case))
    return {"bytes": int(rows * case["vocab"] * size) + sum(_drafts(case)) * (2 * size + 8), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _value_of(code):
    """The value of E4M3 codes (bytes as whole numbers): sign, four exponent bits of bias 7, three mantissa bits."""
    sign = 1.0 - 2.0 * (code >> 7).double()
    e, m = ((code >> 3) & 15).double(), (code & 7).double()
    return sign * torch.where(e > 0, torch.exp2(e - 7.0) * (1.0 + m / 8.0), m * 2.0 ** -9)


def _row64(cache, block, offset):
    """64-bit rows at (block, offset)."""
    row = cache[block, offset]
    if cache.dtype != torch.uint8:
        return row.double()
    scale = row[:, DC + 2 * DR:].contiguous().view(torch.float32).double()
    latent = _value_of(row[:, :DC].long()).view(-1, 4, DC // 4) * scale.unsqueeze(2)
    return torch.cat([latent.reshape(-1, DC), row[:, DC:DC + 2 * DR].contiguous().view(torch.bfloat16).double()], 1)


def _sequence64(s, i, n):
    bs = s["cache"].shape[1]
    t = torch.arange(n, device=DEV)
    return _row64(s["cache"], s["tables"][i].long()[t // bs], t % bs)


def _nearest_code_value(y):
    """The nearest E4M3 value to each |y| <= 448, ties to the even mantissa."""
    e = torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -6)))
    step = torch.exp2(torch.clamp(e, max=8.0) - 3.0)
    return torch.round(y / step) * step


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "write":
        slots = s["slots"]
        rows = [i for i, x in enumerate(slots.tolist()) if x >= 0]
        at = slots[rows]
        if case["cache"] != "fp8":
            flat = torch.zeros(s["cache"].shape[0] * s["cache"].shape[1], DC + DR, dtype=torch.float64, device=DEV)
            flat[at, :DC] = s["latent"][rows].double()
            flat[at, DC:] = s["rope"][rows].double()
            return flat.view(s["cache"].shape)
        nb, bs = s["cache"].shape[:2]
        x = s["latent"][rows].double().view(-1, 4, DC // 4)
        top = x.abs().amax(dim=2)
        e = torch.where(top > 0, torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0)), -100.0)
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)      # log2 next to a power of two
        e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(-100, 119)
        held = [torch.zeros(nb * bs, w, dtype=torch.float64, device=DEV) for w in (DC, DR, 4)]
        held[0][at] = _nearest_code_value(x * torch.exp2(-e).unsqueeze(2)).view(-1, DC)
        held[1][at] = s["rope"][rows].double()
        held[2][at] = torch.exp2(e)
        return [t.view(nb, bs, -1) for t in held]
    if op == "read":
        return torch.cat([_sequence64(s, i, n) for i, n in enumerate(_lens(case))])
    if op == "absorbed":
        t, got = case["new"], []
        for i, n in enumerate(_lens(case)):
            kv = _sequence64(s, i, n)
            for j in range(t):
                seen = kv[:n - t + j + 1]
                got.append(torch.softmax(s["query"][i * t + j].double() @ seen.T * s["scale"], 1) @ seen[:, :DC])
        return torch.stack(got)
    if op == "expanded":
        got, q0, k0 = [], s["query_start"].tolist(), s["kv_start"].tolist()
        for i, n in enumerate(_news(case)):
            lk = k0[i + 1] - k0[i]
            hide = torch.ones(n, lk, dtype=torch.bool, device=DEV).triu(lk - n + 1)
            k, v, q = (s[x][o[i]:o[i + 1]].double() for x, o in (("k_nope", k0), ("value", k0), ("query", q0)))
            r = s["k_rope"][k0[i]:k0[i + 1]].double()
            heads = [torch.softmax(((q[:, a] @ torch.cat([k[:, a], r], 1).T) * s["scale"]).masked_fill(hide, -math.inf), 1)
                     @ v[:, a] for a in range(case["heads"])]
            got.append(torch.stack(heads, 1))
        return torch.cat(got)
    starts, drafts = s["start"].tolist(), s["drafts"].tolist()
    u, pick = s["uniform"].double().tolist(), s["pick"].double().tolist()
    kept, tokens = [], np.full((case["seqs"], case["drafts"] + 1), -1, dtype=np.int32)
    for i in range(case["seqs"]):
        a, n = 0, starts[i + 1] - starts[i]
        while a < n:
            r, d = starts[i] + a, drafts[starts[i] + a]
            if not u[r] * float(s["draft"][r, d]) < float(s["target"][r + i, d]):
                break
            tokens[i, a] = d
            a += 1
        w = s["target"][starts[i] + i + a].double().cpu().numpy()
        if a < n:
            w = np.maximum(w - s["draft"][starts[i] + a].double().cpu().numpy(), 0.0)
        c = np.cumsum(w)
        tokens[i, a] = int(np.searchsorted(c, pick[i] * c[-1], side="right"))
        kept.append(a)
    return [np.array(kept, dtype=np.int32), tokens]
