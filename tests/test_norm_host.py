"""What the norm's calls and the rows' quantiser refuse (no GPU needed)."""
import ctypes

import pytest
import torch

import combine_topk_ids_02_amd as moe

FAKE = ctypes.c_void_p(0x10000)  # never followed: the calls are refused, or have no rows
OFF = ctypes.c_void_p(0x10008)


def shape(T=0, H=512, E=1, R=1, k=1, align=1, block=0):
    return moe.MoeShape(T, H, E, R, k, align, block)


def norm(s=None, **kw):
    a = dict(stream=1, x=FAKE, residual=FAKE, sum=FAKE, wtype=0, weight=FAKE, eps=1e-6, out=FAKE,
             format=0, q=None, q_scale=None, inv=FAKE)
    a.update(kw)
    return moe.lib().moe_norm(s or shape(), *a.values(), None)


def backward(s=None, **kw):
    a = dict(stream=1, d_out=FAKE, sum=FAKE, inv=FAKE, wtype=0, weight=FAKE, d_sum=FAKE, d_x=FAKE,
             d_res=FAKE, d_weight=None, ws=None, room=0)
    a.update(kw)
    return moe.lib().moe_norm_backward(s or shape(), *a.values(), None)


def quant(s=None, **kw):
    a = dict(rows=FAKE, pair_row=FAKE, cap=64, q=FAKE, scale=FAKE, err=None)
    a.update(kw)
    return moe.lib().moe_quantise_rows(s or shape(), *a.values(), None)


BAD = [dict(T=-1), dict(H=0), dict(H=12), dict(H=(1 << 16) + 8), dict(E=0), dict(k=0), dict(k=17),
       dict(align=0), dict(align=2, block=2), dict(T=1 << 30)]


@pytest.mark.parametrize("bad", BAD)
def test_shapes(bad):
    for call in (norm, backward, quant):
        assert call(shape(**bad)) == moe.MOE_ERR_ARG
    assert moe.lib().moe_norm_workspace_bytes(shape(**bad)) == 0


def test_norm_arguments():
    int8 = dict(format=4, q=FAKE, q_scale=FAKE)
    mx = dict(format=1, q=FAKE, q_scale=FAKE)
    for good in ({}, int8, mx, dict(out=None, **int8), dict(residual=None, sum=None),
                 dict(stream=0, wtype=1), dict(inv=None)):
        assert norm(**good) == moe.MOE_OK, good  # no rows: every check passed, nothing launched
    for bad in (dict(stream=2), dict(stream=-1), dict(wtype=2), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(format=2, q=FAKE,
                                                                     q_scale=FAKE),
                dict(format=3, q=FAKE, q_scale=FAKE), dict(out=None), dict(q=FAKE),
                dict(format=4, q=FAKE), dict(format=4, q_scale=FAKE), dict(q_scale=FAKE),
                dict(residual=None), dict(sum=None), dict(x=OFF), dict(residual=OFF),
                dict(sum=OFF), dict(weight=OFF), dict(out=OFF),
                dict(format=4, q=OFF, q_scale=FAKE),
                dict(format=4, q=FAKE, q_scale=ctypes.c_void_p(0x10002)),
                dict(inv=ctypes.c_void_p(0x10002))):
        assert norm(shape(T=4), **bad) == moe.MOE_ERR_ARG, bad
    assert norm(shape(H=1 << 15)) == moe.MOE_OK and norm(shape(H=(1 << 15) + 8)) == moe.MOE_ERR_ARG
    assert norm(shape(H=48), **mx) == moe.MOE_ERR_ARG and norm(shape(H=48), **int8) == moe.MOE_OK
    for bad in (dict(x=None), dict(weight=None)):
        assert norm(shape(T=4), **bad) == moe.MOE_ERR_ARG


def test_backward_arguments():
    need = moe.lib().moe_norm_workspace_bytes(shape(T=600))
    assert need == 512 * 512 * 4
    assert moe.norm_workspace_bytes(3, 5120) == 3 * 5120 * 4
    for good in ({}, dict(d_x=None), dict(d_res=None), dict(d_sum=None), dict(stream=0)):
        assert backward(**good) == moe.MOE_OK, good
    for bad in (dict(stream=2), dict(wtype=2), dict(d_x=None, d_res=None), dict(d_out=OFF),
                dict(sum=OFF), dict(weight=OFF), dict(d_sum=OFF), dict(d_x=OFF), dict(d_res=OFF),
                dict(ws=OFF), dict(inv=ctypes.c_void_p(0x10002)),
                dict(d_weight=ctypes.c_void_p(0x10002), ws=FAKE, room=1 << 30)):
        assert backward(shape(T=4), **bad) == moe.MOE_ERR_ARG, bad
    some = shape(T=600)
    for bad in (dict(d_out=None), dict(sum=None), dict(inv=None), dict(weight=None),
                dict(d_weight=FAKE), dict(d_weight=FAKE, ws=FAKE, room=need - 1),
                dict(d_weight=FAKE, ws=None, room=need)):
        assert backward(some, **bad) == moe.MOE_ERR_ARG, bad


def test_quantiser_arguments():
    some = shape(T=64)
    assert quant() == moe.MOE_OK and quant(cap=0) == moe.MOE_OK
    for bad in (dict(cap=-1), dict(pair_row=None, cap=63), dict(rows=None), dict(q=None),
                dict(scale=None), dict(rows=OFF), dict(q=OFF),
                dict(scale=ctypes.c_void_p(0x10002)), dict(pair_row=ctypes.c_void_p(0x10002))):
        assert quant(some, **bad) == moe.MOE_ERR_ARG, bad


def test_binding_refuses_tensors_of_the_host():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.norm(x, w, out=x)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.norm_backward(x, x, torch.zeros(4), w, d_x=x)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.quantise_rows(x, x.to(torch.int8), torch.zeros(4))
