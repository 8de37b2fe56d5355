"""The latent-cache and verification calls on a machine without a GPU: what
they refuse before any launch, and pins of the plain forms their GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import latent_ref as R
import paged_kv_cache_12_gb300 as pa

NUL = None
FAKE = ctypes.c_void_p(1 << 20)   # an aligned address that no refused call reads
ODD = ctypes.c_void_p((1 << 20) + 8)


def test_write_refusals():
    W = pa.lib().pa_latent_write

    def w(latent=FAKE, rope=FAKE, slots=FAKE, cache=FAKE, n=3, sl=512, sr=64, bs=16, nb=4, kv=pa.PA_KV_BF16):
        return W(latent, rope, slots, cache, n, sl, sr, bs, nb, kv, NUL)
    assert w(n=0) == pa.PA_OK
    assert w(n=0, latent=NUL, rope=NUL, slots=NUL, cache=NUL) == pa.PA_OK
    for bad in (dict(n=-1), dict(nb=0), dict(bs=0), dict(kv=3), dict(kv=-1), dict(sl=511), dict(sl=516), dict(sr=56),
                dict(sr=68), dict(latent=NUL), dict(rope=NUL), dict(slots=NUL), dict(cache=NUL), dict(latent=ODD),
                dict(rope=ODD), dict(cache=ODD)):
        assert w(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert w(bs=24) == pa.PA_ERR_UNSUPPORTED and w(bs=128) == pa.PA_ERR_UNSUPPORTED


def test_copy_and_read_refusals():
    C, G = pa.lib().pa_latent_block_copy, pa.lib().pa_latent_read
    assert C(NUL, NUL, 0, 16, 4, pa.PA_KV_F16, NUL) == pa.PA_OK
    assert C(NUL, FAKE, 1, 16, 4, pa.PA_KV_F16, NUL) == pa.PA_ERR_INVALID_ARG
    assert C(FAKE, FAKE, 1, 16, 4, 7, NUL) == pa.PA_ERR_INVALID_ARG
    assert C(FAKE, FAKE, 1, 12, 4, pa.PA_KV_F16, NUL) == pa.PA_ERR_UNSUPPORTED
    assert C(FAKE, FAKE, 65536, 16, 4, pa.PA_KV_F16, NUL) == pa.PA_ERR_UNSUPPORTED

    def g(out=FAKE, cache=FAKE, tab=FAKE, start=FAKE, b=2, n=5, so=576, bs=16, nb=4, mb=3, kv=pa.PA_KV_FP8_E4M3):
        return G(out, cache, tab, start, NUL, b, n, so, bs, nb, mb, kv, NUL)
    assert g(n=0) == pa.PA_OK and g(n=0, b=0) == pa.PA_OK
    for bad in (dict(out=NUL), dict(cache=NUL), dict(tab=NUL), dict(start=NUL), dict(b=-1), dict(n=-1), dict(b=0),
                dict(so=568), dict(so=580), dict(nb=0), dict(mb=0), dict(kv=4), dict(out=ODD), dict(cache=ODD)):
        assert g(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert g(bs=10) == pa.PA_ERR_UNSUPPORTED


def test_attention_refusals():
    A = pa.lib().pa_latent_attention

    def f(out=FAKE, q=FAKE, cache=FAKE, tab=FAKE, lens=FAKE, qs=NUL, b=2, nq=2, h=16, bs=16, nb=9, mb=4, mx=60, sc=0.1,
          kv=pa.PA_KV_BF16, ws=FAKE, size=1 << 40):
        return A(out, q, cache, tab, lens, qs, b, nq, h, bs, nb, mb, mx, sc, kv, ws, size, NUL)
    assert f(b=0, nq=0) == pa.PA_OK and f(b=3, nq=0, qs=FAKE) == pa.PA_OK
    for bad in (dict(b=-1, nq=-1), dict(nq=3), dict(b=0, nq=1, qs=FAKE), dict(h=0), dict(nb=0), dict(mb=0), dict(mx=-1),
                dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")), dict(sc=float("inf")), dict(kv=9), dict(out=NUL),
                dict(q=NUL), dict(cache=NUL), dict(tab=NUL), dict(lens=NUL), dict(q=ODD), dict(out=ODD),
                dict(cache=ODD)):
        assert f(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(h=129), dict(bs=4), dict(nb=1 << 40)):
        assert f(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=NUL), dict(ws=ctypes.c_void_p((1 << 20) + 128)), dict(size=16)):
        assert f(**bad) == pa.PA_ERR_WORKSPACE, bad
    size = pa.lib().pa_latent_attention_workspace_size
    assert size(1, 1, 0, 10) == 0 and size(1, 1, 129, 10) == 0 and size(-1, 1, 8, 10) == 0 and size(1, 1, 8, -1) == 0
    with pytest.raises(pa.PAError):
        pa.pa_latent_attention_workspace_size(1, 1, 0, 10)


def test_expanded_refusals():
    A = pa.lib().pa_latent_attention_expanded

    def f(out=FAKE, q=FAKE, k=FAKE, r=FAKE, v=FAKE, qs=FAKE, ks=FAKE, b=2, nq=4, nk=9, h=4, kt=512, kh=128, rs=64,
          vt=512, vh=128, sc=0.1, dt=pa.PA_KV_F16, ws=FAKE, size=1 << 40):
        return A(out, q, k, r, v, qs, ks, b, nq, nk, h, kt, kh, rs, vt, vh, sc, dt, ws, size, NUL)
    assert f(nq=0) == pa.PA_OK and f(b=0, nq=0, nk=0) == pa.PA_OK
    for bad in (dict(b=-1), dict(b=0), dict(nq=-1), dict(nk=-1), dict(h=0), dict(kt=120), dict(kh=64), dict(rs=32),
                dict(vt=0), dict(vh=8), dict(kt=516), dict(rs=66), dict(vh=132), dict(sc=0.0), dict(sc=float("nan")),
                dict(dt=pa.PA_KV_FP8_E4M3), dict(out=NUL), dict(q=NUL), dict(k=NUL), dict(r=NUL), dict(v=NUL),
                dict(qs=NUL), dict(ks=NUL), dict(k=ODD), dict(v=ODD), dict(r=ODD), dict(q=ODD), dict(out=ODD)):
        assert f(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(ws=NUL), dict(ws=ctypes.c_void_p((1 << 20) + 64)), dict(size=8)):
        assert f(**bad) == pa.PA_ERR_WORKSPACE, bad
    assert pa.lib().pa_latent_attention_expanded_workspace_size(1, 1, 0) == 0


def test_verify_refusals():
    V = pa.lib().pa_verify_drafts

    def f(acc=FAKE, tok=FAKE, p=FAKE, q=FAKE, d=FAKE, st=FAKE, u=FAKE, s=FAKE, b=2, nd=3, md=2, v=50, ps=50, qs=50, dt=0):
        return V(acc, tok, p, q, d, st, u, s, b, nd, md, v, ps, qs, dt, NUL)
    assert f(b=0, nd=0) == pa.PA_OK
    for bad in (dict(b=-1), dict(b=0), dict(nd=-1), dict(md=-1), dict(v=0), dict(ps=49), dict(qs=49), dict(dt=3),
                dict(acc=NUL), dict(tok=NUL), dict(p=NUL), dict(d=NUL), dict(st=NUL), dict(u=NUL), dict(s=NUL),
                dict(p=ctypes.c_void_p((1 << 20) + 2))):
        assert f(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert f(v=(1 << 30) + 1, ps=1 << 31, qs=1 << 31) == pa.PA_ERR_UNSUPPORTED


def test_bindings_refuse_other_tensors():
    bf, f16 = torch.bfloat16, torch.float16
    with pytest.raises(ValueError):   # not a latent row
        pa.pa_latent_write(torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf),
                           torch.zeros(1, dtype=torch.int64), torch.zeros(2, 16, 640, dtype=torch.uint8))
    with pytest.raises(ValueError):   # host tensors
        pa.pa_latent_write(torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf),
                           torch.zeros(1, dtype=torch.int64), torch.zeros(2, 16, 576, dtype=bf))
    with pytest.raises(ValueError):
        pa.pa_verify_drafts(*[torch.zeros(1)] * 2, torch.zeros(1, 4, dtype=torch.float64), None, *[torch.zeros(1)] * 4)
    with pytest.raises(ValueError):
        pa.pa_latent_attention_expanded(*[torch.zeros(1, 1, 192)] * 5, *[torch.zeros(2)] * 2, 0.1, torch.zeros(1))
    with pytest.raises(ValueError):
        pa.pa_latent_read(torch.zeros(1, 576, dtype=f16), torch.zeros(2, 576, dtype=f16), None, None)


def test_plain_codes():
    # the encoder returns every finite code of its own value, saturates, and
    # breaks ties to the even code; scales hold their group exactly
    c = torch.arange(256, dtype=torch.uint8)
    finite = (c & 127) != 127
    v = R.e4m3_value(c)
    assert torch.equal(R.encode_e4m3(v[finite]), c[finite])
    y = torch.tensor([449.0, 1e9, -464.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10], dtype=torch.float64)
    assert R.encode_e4m3(y).tolist() == [0x7e, 0x7e, 0xfe, 0x38, 0x3a, 0x00, 0x02]
    x = torch.zeros(5, 512, dtype=torch.bfloat16)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 448.0, 450.0, 2.0 ** -120, float(torch.finfo(torch.bfloat16).max)
    _, s = R.quantise(x)
    assert s[:, 0].tolist() == [1.0, 2.0, 2.0 ** -100, 2.0 ** 119, 2.0 ** -100]


def test_plain_verification_distribution():
    # whatever the draft's distribution, the first token comes out as p says
    rng = np.random.default_rng(3)
    p, q = np.array([0.5, 0.2, 0.3]), np.array([0.1, 0.8, 0.1])
    n, count = 20000, np.zeros(3)
    d = rng.choice(3, size=n, p=q)
    u, pick = rng.random(n), rng.random(n)
    target = np.tile(p, (2 * n, 1))
    _, tokens = R.verify(target, np.tile(q, (n, 1)), d, list(range(n + 1)), u, pick, 1)
    for v in range(3):
        count[v] = (tokens[:, 0] == v).mean()
    # five standard deviations of a share over n draws
    assert (np.abs(count - p) <= 5 * np.sqrt(p * (1 - p) / n)).all(), count
