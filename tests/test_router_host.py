"""The router, balance and expert calls refuse bad arguments before anything is
launched (no GPU needed), and the 64-bit formulas the GPU tests compare with
are themselves checked against differences."""
import ctypes

import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe
import router_ref as ref

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(0x10001)
ARG = moe.MOE_ERR_ARG


def shape(T=64, H=512, E=16, R=4, k=2, align=1, block=0):
    return moe.MoeShape(T, H, E, R, k, align, block)


def sigmoid(**kw):
    return moe.Router("sigmoid", **kw)


def route(sh=None, r=None, typ=0, z=FAKE, bias=None, mask=None, ids=FAKE, w=FAKE):
    return moe.lib().moe_route(sh or shape(), ctypes.byref(r or moe.Router()), typ, z, bias, mask,
                               ids, w, None, None)


def backward(sh=None, r=None, typ=0, z=FAKE, ids=FAKE, dw=FAKE, dl=None, counts=FAKE,
             tokens=FAKE, off=None, S=1, dz=FAKE):
    return moe.lib().moe_route_backward(sh or shape(), ctypes.byref(r or moe.Router()), typ, z,
                                        ids, dw, dl, counts, tokens, off, S, dz, None, None)


def balance(sh=None, r=None, typ=0, z=FAKE, ids=FAKE, off=None, S=1, loss=FAKE, counts=FAKE,
            tokens=FAKE, mean=FAKE, ws=FAKE, wsb=1 << 30):
    return moe.lib().moe_balance_loss(sh or shape(), ctypes.byref(r or moe.Router()), typ, z, ids,
                                      off, S, loss, counts, tokens, mean, ws, wsb, None, None)


def product(sh=None, N=64, fmt=2, act=0, rows=FAKE, counts=FAKE, off=FAKE, cap=128, q=FAKE,
            s=FAKE, factor=None, out=FAKE):
    return moe.lib().moe_expert_product(sh or shape(), N, fmt, act, rows, counts, off, cap, q, s,
                                        factor, out, None, None)


BAD_SHAPES = [dict(T=-1), dict(E=0), dict(R=0), dict(E=10, R=4), dict(k=0), dict(k=17, E=64),
              dict(E=2048, R=8), dict(T=1 << 28, k=8)]


@pytest.mark.parametrize("bad", BAD_SHAPES)
def test_bad_shapes(bad):
    s = shape(**bad)
    assert route(s) == ARG and backward(s) == ARG and balance(s) == ARG and product(s) == ARG
    assert moe.lib().moe_balance_workspace_bytes(s, 1) == 0


def test_bad_routers():
    bad = [sigmoid(groups=0), sigmoid(groups=3), sigmoid(groups=128), sigmoid(top_groups=0),
           sigmoid(groups=4, top_groups=5), moe.Router("softmax", groups=4, top_groups=2),
           moe.Router(scale=float("nan")), moe.Router(scale=float("inf"))]
    odd = moe.Router()
    odd.scoring = 2
    bad.append(odd)
    odd = moe.Router()
    odd.renorm = 2
    bad.append(odd)
    for r in bad:
        s = shape(E=128, R=4)
        assert route(s, r) == ARG and backward(s, r) == ARG and balance(s, r) == ARG
    for typ in (-1, 3):
        assert route(typ=typ) == ARG and backward(typ=typ) == ARG and balance(typ=typ) == ARG
    with pytest.raises(moe.MoeError):
        moe.Router("softplus")


def test_route_arguments():
    for kw in (dict(z=None), dict(ids=None), dict(w=None), dict(z=ODD), dict(ids=ODD),
               dict(w=ODD), dict(bias=ODD, r=sigmoid()), dict(bias=FAKE),
               dict(z=ODD, typ=1)):
        assert route(**kw) == ARG, kw
    assert route(shape(T=0), z=None, ids=None, w=None) == moe.MOE_OK  # nothing to do


def test_backward_arguments():
    for kw in (dict(z=None), dict(ids=None), dict(dz=None), dict(dw=None), dict(dz=ODD),
               dict(dl=FAKE, counts=None), dict(dl=FAKE, tokens=None), dict(dl=FAKE, S=0),
               dict(dl=FAKE, S=2), dict(dl=FAKE, S=(1 << 16) + 1, off=FAKE), dict(dl=ODD),
               dict(dl=FAKE, off=ODD), dict(dw=ODD)):
        assert backward(**kw) == ARG, kw
    assert backward(shape(T=0), z=None, ids=None, dz=None) == moe.MOE_OK


def test_balance_arguments():
    need = moe.balance_workspace_bytes(64, 16, 2, 1)
    assert need >= 2 * 16 * 8
    for kw in (dict(z=None), dict(ids=None), dict(loss=None), dict(counts=None),
               dict(tokens=None), dict(mean=None), dict(ws=None), dict(S=0), dict(S=2),
               dict(S=(1 << 16) + 1, off=FAKE), dict(wsb=need - 1), dict(ws=ODD),
               dict(off=ODD)):
        assert balance(**kw) == ARG, kw
    assert moe.balance_workspace_bytes(64, 16, 2, 0) == 0
    assert moe.balance_workspace_bytes(64, 16, 2, 1 << 17) == 0


def test_product_arguments():
    for kw in (dict(N=0), dict(N=(1 << 24) + 1), dict(fmt=0), dict(fmt=1), dict(fmt=4),
               dict(act=2), dict(act=-1), dict(N=63, act=1), dict(rows=None), dict(out=None),
               dict(counts=None), dict(off=None), dict(q=None), dict(s=None), dict(cap=-1),
               dict(rows=ctypes.c_void_p(0x10008)), dict(out=ctypes.c_void_p(0x10002)),
               dict(q=ctypes.c_void_p(0x10004)), dict(s=ODD), dict(factor=ODD),
               dict(sh=shape(H=520)), dict(sh=shape(H=16))):
        assert product(**kw) == ARG, kw
    assert product(shape(T=0), rows=None, out=None, counts=None, off=None, q=None, s=None) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Host tensors, wrong types and shapes raise before any pointer is passed."""
    z = torch.zeros(4, 16)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.route(z, 2, moe.Router(), ids, w)
    with pytest.raises(moe.MoeError, match="logits"):
        moe.route(z.double(), 2, moe.Router(), ids, w)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.route_backward(z, ids, moe.Router(), torch.zeros_like(z), d_weights=w)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.balance_loss(z, ids, moe.Router(), w[0], ids, ids[0], w, workspace=z)
    rows = torch.zeros(8, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 32, dtype=torch.uint8)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.expert_product("mxfp4", rows, ids, ids, 4, 2, q, q, rows)
    with pytest.raises(moe.MoeError, match="format"):
        moe.expert_product("mxfp8", rows, ids, ids, 4, 2, q, q, rows)
    with pytest.raises(moe.MoeError, match="activation"):
        moe.expert_product("mxfp4", rows, ids, ids, 4, 2, q, q, rows, act="gelu")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_against_differences(scoring, renorm):
    """The gradient's formula against central differences of the forward
    formulas: with h = 1e-5 in 64 bits the differences are off by about
    h^2 = 1e-10 and 1e-16 / h = 1e-11, times terms of size 1."""
    rng = np.random.default_rng(3)
    T, E, k = 9, 12, 4
    z = rng.normal(size=(T, E))
    ids, _ = ref.choose(z, k, scoring)
    ids[3] = -1
    ids[4, 2:] = -1
    ids[5, 1] = ids[5, 0]  # the same expert twice
    dw = rng.normal(size=(T, k))
    off = [1, 4, 4, 8]
    dl = rng.normal(size=3)

    def value(z):
        loss, _, _, _ = ref.balance(z, ids, scoring, off)
        return ((ref.weights(z, ids, scoring, renorm, 2.5) * dw).sum() + (loss * dl).sum())

    d, _ = ref.gradient(z, ids, scoring, renorm, 2.5, dw, dl, off)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((value(a) - value(b)) / (2 * h) - d[t, e]) < 1e-8, (t, e)
