"""Calls at the edges of what the router, the balance loss and the expert
products take, refused without a GPU."""
import ctypes

import pytest
import torch

import combine_topk_ids_02_amd as moe

FAKE = ctypes.c_void_p(0x10000)  # never followed: the calls are refused


def test_too_many_tokens():
    """A launch has fewer than 2^32 threads: 2^25 tokens at most."""
    lib = moe.lib()
    s = moe.MoeShape((1 << 25) + 1, 8, 16, 1, 2)
    r = ctypes.byref(moe.Router())
    assert lib.moe_route(s, r, 0, FAKE, None, None, FAKE, FAKE, None, None) == moe.MOE_ERR_ARG
    assert lib.moe_route_backward(s, r, 0, FAKE, FAKE, FAKE, None, None, None, None, 0, FAKE,
                                  None, None) == moe.MOE_ERR_ARG
    assert lib.moe_balance_loss(s, r, 0, FAKE, FAKE, None, 1, FAKE, FAKE, FAKE, FAKE, FAKE,
                                1 << 40, None, None) == moe.MOE_ERR_ARG


def test_missing_workspace():
    z = torch.zeros(4, 16, device="meta")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="meta")
    w = torch.zeros(4, 2, device="meta")
    with pytest.raises(moe.MoeError):
        moe.balance_loss(z, ids, moe.Router(), w[0], ids, ids[0], w, workspace=None)
