"""The calls of a step over a tree (write with rotation, tree attention, tree
verification, move of the path) on a machine without a GPU: what they refuse
before any launch, and pins of the plain forms their GPU tests use."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_12_gb300 as pa
import tree_ref as TR

NUL = None
FAKE = ctypes.c_void_p(1 << 20)   # an aligned address that no refused call reads
OTHER = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 8)
NAN, INF = float("nan"), float("inf")


def test_rope_refusals():
    W = pa.lib().pa_kv_write_rope

    def w(qo=OTHER, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, inv=FAKE, ax=NUL, slots=FAKE, kc=FAKE, vc=FAKE, n=3, hq=8, hk=2,
          d=64, r=64, axes=1, il=0, sq=512, so=512, sk=128, sv=128, bs=16, nb=4, kv=pa.PA_KV_BF16, ks=1.0, vs=1.0):
        return W(qo, q, k, v, pos, inv, ax, slots, kc, vc, n, hq, hk, d, r, axes, il, sq, so, sk, sv, bs, nb, kv, ks,
                 vs, NUL)
    assert w(n=0) == pa.PA_OK
    assert w(n=0, q=NUL, qo=NUL, k=NUL, v=NUL, pos=NUL, inv=NUL, slots=NUL, kc=NUL, vc=NUL) == pa.PA_OK
    assert w(n=0, hq=0, sq=0, so=0) == pa.PA_OK
    for bad in (dict(n=-1), dict(hq=-1), dict(hk=0), dict(d=0), dict(d=60), dict(r=0), dict(r=8), dict(r=72),
                dict(r=80), dict(axes=0), dict(axes=5), dict(bs=0), dict(nb=0), dict(kv=3), dict(kv=-1), dict(sq=504),
                dict(so=504), dict(sk=120), dict(sv=64), dict(sq=516), dict(so=514), dict(sk=132), dict(sv=129),
                dict(k=NUL), dict(v=NUL), dict(pos=NUL), dict(inv=NUL), dict(slots=NUL), dict(kc=NUL), dict(vc=NUL),
                dict(q=NUL), dict(qo=NUL), dict(k=ODD), dict(v=ODD), dict(kc=ODD), dict(vc=ODD), dict(q=ODD),
                dict(qo=ODD), dict(qo=FAKE, so=520),
                dict(kv=pa.PA_KV_FP8_E4M3, ks=0.0), dict(kv=pa.PA_KV_FP8_E4M3, vs=-1.0),
                dict(kv=pa.PA_KV_FP8_E4M3, ks=NAN), dict(kv=pa.PA_KV_FP8_E4M3, vs=INF)):
        assert w(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert w(d=1024, r=528, sq=8192, so=8192, sk=2048, sv=2048) == pa.PA_ERR_UNSUPPORTED


def test_tree_attention_refusals():
    A = pa.lib().pa_attention_tree

    def f(out=FAKE, q=FAKE, k=FAKE, v=FAKE, tab=FAKE, lens=FAKE, qs=FAKE, par=FAKE, b=2, nq=9, hq=8, hk=2, d=128,
          bs=16, nb=9, mb=4, mx=60, sc=0.1, kv=pa.PA_KV_F16, ks=1.0, vs=1.0, ws=FAKE, size=1 << 40):
        return A(out, q, k, v, tab, lens, qs, par, b, nq, hq, hk, d, bs, nb, mb, mx, sc, kv, ks, vs, ws, size, NUL)
    assert f(nq=0) == pa.PA_OK and f(b=0, nq=0) == pa.PA_OK
    for bad in (dict(b=-1), dict(b=0), dict(nq=-1), dict(hq=0), dict(hk=0), dict(hq=9), dict(nb=0), dict(mb=0),
                dict(mx=-1), dict(sc=0.0), dict(sc=-1.0), dict(sc=NAN), dict(sc=INF), dict(kv=9), dict(out=NUL),
                dict(q=NUL), dict(k=NUL), dict(v=NUL), dict(tab=NUL), dict(lens=NUL), dict(qs=NUL), dict(par=NUL),
                dict(out=ODD), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(kv=pa.PA_KV_FP8_E4M3, ks=0.0),
                dict(kv=pa.PA_KV_FP8_E4M3, vs=NAN)):
        assert f(**bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(d=96), dict(bs=64), dict(bs=4), dict(hq=34), dict(nb=1 << 40), dict(kv=pa.PA_KV_FP8_E4M3, d=64),
                dict(nq=(1 << 31) - 1)):
        assert f(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=NUL), dict(ws=ctypes.c_void_p((1 << 20) + 128)), dict(size=16)):
        assert f(**bad) == pa.PA_ERR_WORKSPACE, bad
    size = pa.lib().pa_attention_tree_workspace_size
    assert size(1, 1, 8, 3, 128, 10) == 0 and size(-1, 1, 8, 8, 128, 10) == 0 and size(1, 1, 8, 8, 128, -1) == 0
    assert size(1, 8, 64, 8, 128, 600) >= 256
    with pytest.raises(pa.PAError):
        pa.pa_attention_tree_workspace_size(1, 1, 0, 1, 128, 10)


def test_verify_tree_refusals():
    V = pa.lib().pa_verify_tree

    def f(acc=FAKE, tok=FAKE, path=FAKE, p=FAKE, d=FAKE, par=FAKE, st=FAKE, u=FAKE, b=2, n=7, md=2, v=50, ps=50, dt=0):
        return V(acc, tok, path, p, d, par, st, u, b, n, md, v, ps, dt, NUL)
    assert f(b=0, n=0) == pa.PA_OK
    for bad in (dict(b=-1), dict(b=0), dict(n=-1), dict(md=-1), dict(v=0), dict(ps=49), dict(dt=3), dict(acc=NUL),
                dict(tok=NUL), dict(path=NUL), dict(p=NUL), dict(d=NUL), dict(par=NUL), dict(st=NUL), dict(u=NUL),
                dict(p=ctypes.c_void_p((1 << 20) + 2)), dict(p=ctypes.c_void_p((1 << 20) + 1), dt=2)):
        assert f(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert f(v=(1 << 30) + 1, ps=1 << 31) == pa.PA_ERR_UNSUPPORTED


def test_move_path_refusals():
    M = pa.lib().pa_kv_move_path

    def f(k=FAKE, v=FAKE, tab=FAKE, lens=FAKE, qs=FAKE, path=FAKE, acc=FAKE, b=2, md=3, layers=1, hk=2, d=64, bs=16,
          nb=9, mb=4, kv=pa.PA_KV_F16):
        return M(k, v, tab, lens, qs, path, acc, b, md, layers, hk, d, bs, nb, mb, kv, NUL)
    assert f(b=0) == pa.PA_OK and f(md=0) == pa.PA_OK   # node 0 is in its place
    for bad in (dict(b=-1), dict(md=-1), dict(layers=0), dict(hk=0), dict(d=0), dict(d=60), dict(bs=0), dict(nb=0),
                dict(mb=0), dict(kv=5), dict(kv=pa.PA_KV_FP8_E4M3, d=72), dict(k=NUL), dict(v=NUL), dict(tab=NUL),
                dict(lens=NUL), dict(qs=NUL), dict(path=NUL), dict(acc=NUL), dict(k=ODD), dict(v=ODD)):
        assert f(**bad) == pa.PA_ERR_INVALID_ARG, bad


def test_bindings_refuse_other_tensors():
    f16, i32 = torch.float16, torch.int32
    z = torch.zeros
    with pytest.raises(ValueError):   # host tensors
        pa.pa_kv_write_rope(z(1, 1, 64, dtype=f16), z(1, 1, 64, dtype=f16), z(1, dtype=i32), z(32), z(1), z(2, 1, 16, 64, dtype=f16),
                            z(2, 1, 16, 64, dtype=f16))
    with pytest.raises(ValueError):   # no cache type
        pa.pa_kv_write_rope(z(1, 1, 64), z(1, 1, 64), z(1, dtype=i32), z(32), z(1), z(2, 1, 16, 64), z(2, 1, 16, 64))
    with pytest.raises(ValueError):
        pa.pa_attention_tree(z(1, 8, 64), z(1, 8, 64), z(2, 1, 16, 64, dtype=f16), z(2, 1, 16, 64, dtype=f16), z(1, 2), z(1),
                             z(2), z(1), 0.1, 10, z(1))
    with pytest.raises(ValueError):
        pa.pa_verify_tree(z(1), z(1, 2), z(1, 2), z(1, 4, dtype=torch.float64), z(1), z(1), z(2), z(1))
    with pytest.raises(ValueError):
        pa.pa_kv_move_path(z(2, 1, 16, 64, dtype=f16), z(2, 1, 16, 64, dtype=f16), z(1, 2), z(1), z(2), z(1, 2), z(1))


def test_plain_rotation():
    # a quarter turn takes (x, y) to (-y, x); positions add up; lengths stay; the rest of the head stays
    x = torch.randn(3, 2, 48, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    quarter = torch.full((16,), math.pi / 2, dtype=torch.float64)
    one = torch.ones(1, 3, dtype=torch.int32)
    for il in (False, True):
        y = TR.rotate(x, one, quarter, None, il)
        a, b = (slice(0, 32, 2), slice(1, 32, 2)) if il else (slice(0, 16), slice(16, 32))
        assert torch.allclose(y[..., a], -x[..., b], atol=1e-15) and torch.allclose(y[..., b], x[..., a], atol=1e-15)
        assert torch.equal(y[..., 32:], x[..., 32:])
        inv = torch.rand(16, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
        twice = TR.rotate(TR.rotate(x, 5 * one, inv, None, il), 7 * one, inv, None, il)
        assert torch.allclose(twice, TR.rotate(x, 12 * one, inv, None, il), atol=1e-12)
    # each pair goes by its axis
    pos = torch.tensor([[1, 1, 1], [0, 0, 0]], dtype=torch.int32)
    axis = torch.tensor([0, 1] * 8, dtype=torch.int32)
    y = TR.rotate(x, pos, quarter, axis, False)
    assert torch.equal(y[..., 1:16:2], x[..., 1:16:2]) and not torch.equal(y[..., 0:16:2], x[..., 0:16:2])


def test_plain_tree_attention():
    # a chain is the causal mask; a bush's leaves see the root and themselves
    assert torch.equal(TR.ancestors([-1, 0, 1, 2]), torch.ones(4, 4).tril().bool())
    assert TR.ancestors([-1, 0, 0, 1]).tolist() == [[True, False, False, False], [True, True, False, False],
                                                    [True, False, True, False], [True, True, False, True]]
    # identical keys give the mean of what is seen
    v = torch.randn(6, 1, 64, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    sees = torch.tensor([[1, 1, 1, 1, 0, 0], [1, 1, 0, 0, 0, 1]]).bool()
    o, bound = TR.tree_attention(torch.ones(2, 1, 64), torch.ones(6, 1, 64, dtype=torch.float64), v, sees, 0.125,
                                 torch.float16)
    assert torch.allclose(o[0, 0], v[:4, 0].mean(0)) and torch.allclose(o[1, 0], v[[0, 1, 5], 0].mean(0))
    assert (bound > 0).all() and (bound < 0.01).all()


def test_plain_tree_verification_distribution():
    # whatever the children are, the first token comes out as p says, and so does the one after a given first
    rng = np.random.default_rng(5)
    p = np.array([[0.5, 0.2, 0.3], [0.1, 0.6, 0.3], [0.25, 0.25, 0.5]])
    n = 20000
    target = np.tile(p, (n, 1))
    tokens, parents = [0, 1, 0] * n, [-1, 0, 0] * n       # children of the root: tokens 1 (node 1) and 0 (node 2)
    _, out, path = TR.verify_tree(target, tokens, parents, list(range(0, 3 * n + 1, 3)), rng.random(3 * n), 1)
    first = np.array([(out[:, 0] == v).mean() for v in range(3)])
    # five standard deviations of a share over n draws
    assert (np.abs(first - p[0]) <= 5 * np.sqrt(p[0] * (1 - p[0]) / n)).all(), first
    for node, token in ((1, 1), (2, 0)):
        after = out[out[:, 0] == token]
        assert (path[out[:, 0] == token, 1] == node).all()
        share = np.array([(after[:, 1] == v).mean() for v in range(3)])
        assert (np.abs(share - p[node]) <= 5 * np.sqrt(p[node] * (1 - p[node]) / len(after))).all(), share
    assert (out[out[:, 0] == 2, 1] == -1).all()


def test_counts_that_do_not_fit_are_refused():
    # a row of max_depth + 1 tokens, and steps of a warp or more past the end, are counted in 32 bits
    most, V, D = (1 << 31) - 1, pa.lib().pa_verify_tree, pa.lib().pa_verify_drafts
    for n, depth in ((7, most), (most, 2), (7, (1 << 30) + 1), ((1 << 30) + 1, 2)):
        assert V(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, n, depth, 50, 50, 0, NUL) == pa.PA_ERR_UNSUPPORTED
        assert D(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, n, depth, 50, 50, 50, 0, NUL) == pa.PA_ERR_UNSUPPORTED


def test_sizes_of_a_move_that_do_not_fit_are_refused():
    # a sequence's max_depth + 1 path entries and a row's bytes are counted in 32 bits
    M, most = pa.lib().pa_kv_move_path, (1 << 31) - 1
    for md, d in ((most, 64), ((1 << 30) + 1, 64), (3, 1 << 30), (3, most - 7)):
        assert M(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, md, 1, 2, d, 16, 9, 4, pa.PA_KV_F16, NUL) == \
            pa.PA_ERR_UNSUPPORTED, (md, d)
