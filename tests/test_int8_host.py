"""What the products in 8-bit integers refuse (no GPU needed)."""
import ctypes

import pytest
import torch

import combine_topk_ids_02_amd as moe

FAKE = ctypes.c_void_p(0x10000)  # never followed: the calls are refused, or have no rows
OFF = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)


def call(N=64, act=0, T=4, H=512, E=8, R=1, k=2, align=1, block=0, **kw):
    a = dict(rows=FAKE, row_scale=FAKE, counts=FAKE, offsets=FAKE, cap=64, w=FAKE, w_scale=FAKE,
             out=FAKE, err=None)
    a.update(kw)
    return moe.lib().moe_int8_product(moe.MoeShape(T, H, E, R, k, align, block), N, act,
                                      *a.values(), None)


def test_calls_without_rows():
    for good in ({}, dict(act=1), dict(H=16), dict(H=65536), dict(N=1 << 24), dict(N=1),
                 dict(E=1024), dict(rows=None, out=None)):
        assert call(T=0, **good) == moe.MOE_OK, good


@pytest.mark.parametrize("bad", [
    dict(H=8), dict(H=24), dict(H=65552), dict(N=0), dict(N=(1 << 24) + 1), dict(act=2),
    dict(act=-1), dict(N=65, act=1), dict(cap=-1), dict(E=0), dict(E=1025), dict(k=17),
    dict(T=-1), dict(R=3), dict(align=0)])
def test_sizes(bad):
    for T in (0, 4):
        assert call(**{"T": T, **bad}) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(rows=None), dict(row_scale=None), dict(w=None), dict(w_scale=None), dict(out=None),
    dict(counts=None), dict(offsets=None), dict(counts=None, offsets=None),
    dict(counts=None, offsets=None, E=1, cap=7), dict(rows=OFF), dict(w=OFF), dict(out=OFF),
    dict(row_scale=ODD), dict(w_scale=ODD), dict(counts=ODD), dict(offsets=ODD)])
def test_pointers(bad):
    assert call(**bad) == moe.MOE_ERR_ARG


def test_binding():
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    w, ws = torch.zeros(1, 32, 64, dtype=torch.int8), torch.zeros(1, 32)
    out = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.int8_product(q, s, w, ws, out)
    with pytest.raises(moe.MoeError, match="activation"):
        moe.int8_product(q, s, w, ws, out, act="gelu")
