"""The balance loss's workspace and the shapes that the router and product
calls take (no GPU needed)."""
import ctypes
import random

import pytest

import combine_topk_ids_02_amd as moe

FAKE = ctypes.c_void_p(0x10000)  # never followed: the calls are refused


def tiles_of(T):
    """Tiles of one call: 32 tokens each, 64 where that would make more than 64
    tiles, more where even that would make more than 256."""
    if T == 0:
        return 0
    passes = max(2 if T > 2048 else 1, -(-(-(-T // 256)) // 32))
    return -(-T // (32 * passes))


def need(T, E, S):
    return (tiles_of(T) + S) * (-(-E // 4) * 4 * 8 + 4)


def test_balance_workspace_does_not_shrink():
    """A workspace for the largest batch does for every smaller one."""
    most = 0
    last = 0
    for T in range(0, 40000):
        got = moe.balance_workspace_bytes(T, 256, 8, 1)
        most = max(most, need(T, 256, 1))
        assert got == most >= last, T  # what the batches up to T need, and no more
        last = got
    rng = random.Random(5)
    for _ in range(3000):
        T, E, S = rng.randint(0, 1 << 25), rng.randint(2, 1024), rng.randint(1, 1 << 16)
        got = moe.balance_workspace_bytes(T, E, 2, S)
        for t, e, s in ((rng.randint(0, T), rng.randint(2, E), rng.randint(1, S)),
                        (T // 2, E, S), (T, E - 1 or 1, S), (max(T - 1, 0), E, S)):
            assert moe.balance_workspace_bytes(t, e, 1, s) <= got, (T, E, S, t, e, s)
            assert need(t, e, s) <= got


def balance(T, E, S, workspace_bytes):
    s = moe.MoeShape(T, 8, E, 1, 2)
    return moe.lib().moe_balance_loss(s, ctypes.byref(moe.Router()), 0, FAKE, FAKE, FAKE, S, FAKE,
                                      FAKE, FAKE, FAKE, FAKE, workspace_bytes, None, None)


@pytest.mark.parametrize("T", [1, 2048, 2049, 8192, 16384, 16385])
def test_balance_refuses_a_short_workspace(T):
    for S in (1, 7):
        assert balance(T, 64, S, need(T, 64, S) - 1) == moe.MOE_ERR_ARG


def test_shape_of_a_slice_of_the_experts():
    """The products of a slice take a shape of their own: R = 1, whatever the
    layout's R (8 experts of a rank of 32, say), align = 1 and block = 0. Fields
    that change nothing have to keep the limits all the same."""
    def product(**kw):
        s = dict(T=0, H=512, E=8, R=1, k=8, align=1, block=0)
        s.update(kw)
        return moe.lib().moe_expert_product(moe.MoeShape(**s), 64, 2, 0, FAKE, FAKE, FAKE, 64,
                                            FAKE, FAKE, None, FAKE, None, None)

    def route(**kw):
        s = dict(T=0, H=8, E=8, R=1, k=8, align=1, block=0)
        s.update(kw)
        return moe.lib().moe_route(moe.MoeShape(**s), ctypes.byref(moe.Router()), 0, FAKE, None,
                                   None, FAKE, FAKE, None, None)

    for call in (product, route):
        assert call() == moe.MOE_OK  # no tokens: every check passed, nothing launched
        assert call(E=256, R=32) == moe.MOE_OK and call(E=7) == moe.MOE_OK
        for bad in (dict(R=32), dict(R=0), dict(align=0), dict(align=2, block=2), dict(block=-1),
                    dict(H=12)):
            assert call(**bad) == moe.MOE_ERR_ARG, bad
    assert route(H=24) == moe.MOE_OK and product(H=24) == moe.MOE_ERR_ARG
