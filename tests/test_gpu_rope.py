"""pa_kv_write_rope against the rotation in 64 bits (bounds derived in tree_ref.rotation_bound)."""
import numpy as np
import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa
import tree_ref as TR

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
KS, VS = 1 / 50.0, 1 / 30.0   # scales that are no powers of two


def inputs(kv, n, hq, hk, d, pairs, axes=1, bs=16, seed=0, first=0, fused=True, spread=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = TR.ROWS[kv]
    s = {}
    if fused:   # slices of one projection's rows
        rows = torch.randn(n, hq + 2 * hk, d, generator=g, device=DEV).to(dt)
        s["query"], s["key"], s["value"] = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
    else:
        s["query"], s["key"], s["value"] = (torch.randn(n, h, d, generator=g, device=DEV).to(dt) for h in (hq, hk, hk))
    nb = -(-n // bs) + 3
    s["slots"] = torch.randperm(nb * bs, generator=g, device=DEV)[:n]
    s["slots"][5::7] = -1
    s["positions"] = torch.randint(0, spread or max(1, n), (axes, n), generator=g, device=DEV, dtype=torch.int32) + first
    s["inv_freq"] = (10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)).float()
    s["pair_axis"] = torch.randint(0, axes, (pairs,), generator=g, device=DEV, dtype=torch.int32) if axes > 1 else None
    shape = (nb, hk, bs, d)
    if kv == pa.PA_KV_FP8_E4M3:
        s["k_cache"], s["v_cache"] = (torch.full(shape, x, dtype=torch.uint8, device=DEV) for x in (0x31, 0x42))
    else:
        s["k_cache"], s["v_cache"] = (torch.full(shape, x, dtype=dt, device=DEV) for x in (3.0, 5.0))
    return s


def call(s, kv, query_out, interleaved=False, **more):
    scales = dict(k_scale=KS, v_scale=VS) if kv == pa.PA_KV_FP8_E4M3 else {}
    pa.pa_kv_write_rope(s["key"], s["value"], s["positions"], s["inv_freq"], s["slots"], s["k_cache"], s["v_cache"],
                        query=s["query"], query_out=query_out, pair_axis=s["pair_axis"], interleaved=interleaved,
                        **scales, **more)


def check(s, kv, out, untouched, interleaved=False, before=None):
    """Every output element against the 64-bit form; `untouched`: what padding's rows of out held."""
    before = before or s
    dt, args = TR.ROWS[kv], (s["positions"], s["inv_freq"], s["pair_axis"], interleaved)
    real = s["slots"] >= 0
    if out is not None:
        want, bound = TR.rotate(before["query"], *args), TR.rotation_bound(before["query"], *args, dt)
        assert torch.equal(out[~real], untouched[~real])
        off = (out.double() - want).abs()
        assert (off <= bound)[real].all(), (off - bound)[real].max()
    bs = s["k_cache"].shape[2]
    at = s["slots"][real]
    written = torch.zeros(s["k_cache"].shape[0], bs, dtype=torch.bool, device=DEV)
    written[at // bs, at % bs] = True
    want = TR.rotate(before["key"], *args)[real]
    k, v = (c[at // bs, :, at % bs] for c in (s["k_cache"], s["v_cache"]))
    if kv == pa.PA_KV_FP8_E4M3:
        f32 = TR.rotation_bound(before["key"], *args, torch.float32)[real]
        y = want / KS
        slack = f32 / KS + y.abs() * 2.0 ** -22   # the scale's reciprocal and the product, a half step each of fp32
        got = R.e4m3_value(k)
        full = y.abs() + slack >= 448.0
        # half a step of a code, or half a subnormal step (2^-10); saturated beyond 448
        bound = torch.maximum((y.abs() + slack) * 2.0 ** -4, torch.full_like(y, 2.0 ** -10)) + slack
        assert torch.where(full, got.abs() >= 416, (got - y).abs() <= bound).all()
        # values are quantised like pa_kv_write_fp8's
        kc, vc = (torch.zeros_like(s["v_cache"]) for _ in range(2))
        pa.pa_kv_write_fp8(before["value"].contiguous(), before["value"].contiguous(), s["slots"], kc, vc, KS, VS)
        assert torch.equal(v, vc[at // bs, :, at % bs])
        rest = (0x31, 0x42)
    else:
        bound = TR.rotation_bound(before["key"], *args, dt)[real]
        off = (k.double() - want).abs()
        assert (off <= bound).all(), (off - bound).max()
        assert torch.equal(v, before["value"][real])
        rest = (3.0, 5.0)
    for c, x in zip((s["k_cache"], s["v_cache"]), rest):   # other slots stay
        assert (c.transpose(1, 2)[~written] == x).all()


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rope,axes,bs", [
    (1, 8, 1, 64, 64, 1, 16), (3, 5, 1, 128, 128, 1, 8), (37, 12, 4, 96, 96, 3, 32), (100, 64, 8, 128, 128, 1, 16),
    (129, 4, 4, 80, 32, 2, 16), (33, 3, 3, 8 * 19, 16 * 9, 4, 8), (1300, 2, 1, 256, 256, 1, 64), (7, 1, 1, 512, 512, 2, 5),
    (50, 6, 2, 128, 64, 3, 16), (9, 2, 2, 16, 16, 1, 1)])
def test_against_64_bits(kv, interleaved, n, hq, hk, d, rope, axes, bs):
    s = inputs(kv, n, hq, hk, d, rope // 2, axes, bs, seed=n + d)
    out = torch.full_like(s["query"], 7.0).contiguous()
    kept = out.clone()
    call(s, kv, out, interleaved)
    torch.cuda.synchronize()
    check(s, kv, out, kept, interleaved)


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
@pytest.mark.parametrize("first", [131072, 10 ** 6, 2 ** 31 - 200, -(2 ** 31)])
def test_far_positions(kv, first):
    s = inputs(kv, 64, 4, 2, 64, 32, first=first, spread=100, seed=5)
    out = torch.zeros(64, 4, 64, dtype=TR.ROWS[kv], device=DEV)
    kept = out.clone()
    call(s, kv, out)
    check(s, kv, out, kept)


def test_in_place_and_without_queries():
    for fused in (True, False):
        kv = pa.PA_KV_BF16
        s = inputs(kv, 45, 8, 2, 128, 32, fused=fused, seed=9)
        before = {x: s[x].clone() for x in ("query", "key", "value")}
        call(s, kv, None)
        check(s, kv, s["query"], before["query"], before=before)
        assert torch.equal(s["key"], before["key"]) and torch.equal(s["value"], before["value"])
    s = inputs(pa.PA_KV_F16, 20, 1, 3, 64, 32, seed=2)
    s["query"] = None
    call(s, pa.PA_KV_F16, None)
    check(s, pa.PA_KV_F16, None, None)


def test_out_rows_with_a_stride():
    kv = pa.PA_KV_F16
    s = inputs(kv, 21, 4, 2, 64, 32, seed=3)
    wide = torch.full((21, 6, 64), 2.0, dtype=torch.float16, device=DEV)
    out = wide[:, 1:5]
    kept = out.clone()
    call(s, kv, out)
    check(s, kv, out, kept)
    assert (wide[:, 0] == 2).all() and (wide[:, 5] == 2).all()


@pytest.mark.parametrize("kv", R.KVS, ids=R.KV_IDS)
def test_as_pa_kv_write_at_position_zero(kv):
    # a turn by nothing is the write as it was
    s = inputs(kv, 50, 4, 4, 128, 64, seed=4)
    s["positions"].zero_()
    out = torch.zeros(50, 4, 128, dtype=TR.ROWS[kv], device=DEV)
    k2, v2 = s["k_cache"].clone(), s["v_cache"].clone()
    call(s, kv, out)
    key, value = s["key"].contiguous(), s["value"].contiguous()
    if kv == pa.PA_KV_FP8_E4M3:
        pa.pa_kv_write_fp8(key, value, s["slots"], k2, v2, KS, VS)
    else:
        pa.pa_kv_write(key, value, s["slots"], k2, v2)
    assert torch.equal(s["k_cache"], k2) and torch.equal(s["v_cache"], v2)
    real = s["slots"] >= 0
    assert torch.equal(out[real], s["query"][real])


def test_axis_out_of_range_and_slots_past_the_cache():
    kv = pa.PA_KV_F16
    s = inputs(kv, 16, 2, 1, 64, 32, axes=2, seed=6)
    s["pair_axis"][3], s["pair_axis"][9] = 2, -1
    total = s["k_cache"].shape[0] * 16
    s["slots"][0] = total
    s["slots"][1] = 2 ** 40
    out = torch.zeros(16, 2, 64, dtype=torch.float16, device=DEV)
    call(s, kv, out)
    assert (out[:2] == 0).all()
    nan = torch.zeros(64, dtype=torch.bool, device=DEV)
    nan[[3, 9, 35, 41]] = True
    real = (s["slots"] >= 0) & (s["slots"] < total)
    assert torch.isnan(out[real])[..., nan].all() and not torch.isnan(out[real])[..., ~nan].any()


def test_infinities_and_nan_stay_in_their_pairs():
    kv = pa.PA_KV_BF16
    s = inputs(kv, 4, 1, 1, 64, 32, seed=8, fused=False)
    s["slots"][:] = torch.arange(4, device=DEV)
    s["query"][2, 0, 5] = float("nan")
    s["key"][1, 0, 40] = float("inf")
    out = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    call(s, kv, out)
    bad = ~torch.isfinite(out[:, 0])
    assert bad[2, 5] and bad[2, 37] and bad.sum() == 2
    bad = ~torch.isfinite(s["k_cache"][0, 0, :4])
    assert bad[1, 40] and bad[1, 8] and bad.sum() == 2


def test_streams_graphs_and_repeats():
    kv = pa.PA_KV_BF16
    s = inputs(kv, 300, 16, 4, 128, 64, seed=12)
    out = torch.zeros(300, 16, 128, dtype=torch.bfloat16, device=DEV)
    call(s, kv, out)
    torch.cuda.synchronize()
    want, kc, vc = out.clone(), s["k_cache"].clone(), s["v_cache"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_(), s["k_cache"].fill_(3), s["v_cache"].fill_(5)
    side.wait_stream(torch.cuda.current_stream())
    call(s, kv, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(s["k_cache"], kc) and torch.equal(s["v_cache"], vc)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, kv, out)
    out.zero_()
    s["positions"].add_(17)
    graph.replay()
    torch.cuda.synchronize()
    s["k_cache"].fill_(3), s["v_cache"].fill_(5)
    graph.replay()
    check(s, kv, out, torch.zeros_like(out))


def test_refusals():
    kv = pa.PA_KV_F16
    s = inputs(kv, 8, 2, 1, 64, 32, seed=1)
    out = torch.zeros(8, 2, 64, dtype=torch.float16, device=DEV)

    def refused(**change):
        t = {**s, **change}
        with pytest.raises((ValueError, pa.PAError)):
            call(t, kv, change.get("out", out))
    refused(key=s["key"].float())
    refused(key=s["key"][:7])
    refused(value=s["value"].transpose(1, 2))
    refused(query=s["query"].bfloat16())
    refused(positions=s["positions"].long())
    refused(positions=s["positions"][:, :7])
    refused(positions=s["positions"].repeat(5, 1))
    refused(inv_freq=s["inv_freq"].double())
    refused(inv_freq=s["inv_freq"][:31])
    refused(inv_freq=torch.zeros(40, device=DEV))
    refused(pair_axis=torch.zeros(31, dtype=torch.int32, device=DEV))
    refused(slots=s["slots"].int())
    refused(v_cache=s["v_cache"][:-1])
    refused(out=torch.zeros(8, 2, 32, dtype=torch.float16, device=DEV))
    refused(query=None)   # a query_out without queries
