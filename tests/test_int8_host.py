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


def test_the_bindings_cpp_part():
    """It says no to what is not a GPU's tensor, and passes numbers and structures on
    as ctypes does."""
    if moe._fast is None:
        pytest.skip("not built, or built after the package was imported")
    t = torch.zeros(4, 64)
    for args in ((t, torch.float32, 0, (4, 64)), (t, torch.float32, None, (4, 64)),
                 (None, torch.float32, 0, (4, 64)), (t, torch.float32, 0), (3, 4, 5, 6)):
        assert moe._fast.address(*args) is None
    moe.lib()
    shape = moe.MoeShape(0, 64, 1, 1, 1)
    args = [shape, 1, 0x10000, None, None, 0, 0x10000, 1e-6, 0x10000, 0, None, None, None, None]
    assert moe._fast.moe_norm(*args) == moe.MOE_OK == moe.lib().moe_norm(*args)
    for at, bad in ((7, 0.0), (1, 2), (2, 0x10008), (9, 3)):
        wrong = list(args)
        wrong[at] = bad
        assert moe._fast.moe_norm(*wrong) == moe.MOE_ERR_ARG == moe.lib().moe_norm(*wrong)
    for wrong in (args[:-1], args + [None]):
        with pytest.raises(TypeError):
            moe._fast.moe_norm(*wrong)
    for at, bad in ((1, 1 << 40), (1, "1"), (2, 1.5), (7, "x"), (0, object())):
        wrong = list(args)
        wrong[at] = bad
        with pytest.raises((TypeError, OverflowError, BufferError)):
            moe._fast.moe_norm(*wrong)
