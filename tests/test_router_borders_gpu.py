"""Router calls whose values lie at the borders of float32: group scores whose
keys are much larger than their sum."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe
import router_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


def say(msg):
    print(msg, flush=True)


def choose(z, k, router, bias):
    """z [T, E] and bias [E], float32; the ids of moe.route."""
    z_d, b_d = torch.from_numpy(z).cuda(), torch.from_numpy(bias).cuda()
    ids = torch.full((z.shape[0], k), -7, dtype=torch.int32, device="cuda")
    w = torch.zeros(z.shape[0], k, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.route(z_d, k, router, ids, w, bias=b_d, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and bool(torch.isfinite(w).all())
    return ids.cpu().numpy()


def chosen_by_groups(z, k, bias, groups, top_groups):
    """ref.choose for finite biased sigmoid keys, all tokens at once."""
    T, E = z.shape
    key = ref.sigmoid(z).astype(np.float32) + bias
    best = -np.sort(-key.reshape(T, groups, E // groups), axis=2)[:, :, :2]
    total = best[..., 0] + best[..., 1]  # float32
    order = np.argsort(-total, axis=1, kind="stable")
    keep = np.zeros((T, groups), bool)
    np.put_along_axis(keep, order[:, :top_groups], True, axis=1)
    key = np.where(np.repeat(keep, E // groups, axis=1), key, -np.inf)
    return np.argsort(-key, axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("E,groups,top", [(64, 4, 2), (256, 8, 4), (60, 4, 2)])
@pytest.mark.parametrize("size", [8.0, 64.0, 1024.0, 65536.0])
@pytest.mark.parametrize("kind", ["pair", "all"])
def test_group_scores_that_cancel(E, groups, top, size, kind):
    """A group's two best keys are +size and -size and a score each: their sum
    is near 0, but each key was rounded at its own size. Groups whose scores are
    a few such roundings apart (two of them at the border of the choice, or
    all), against the exact keys."""
    say(f"[cancel] E={E} groups={groups} top={top} size={size} {kind}")
    rng = np.random.default_rng(int(size) + E)
    T, per = 40000, E // groups
    bias = np.full((groups, per), -4 * size, np.float32)
    bias[:, 1], bias[:, per - 2] = size, -size
    z = rng.normal(size=(T, groups, per)).astype(np.float32)
    if kind == "pair":  # one in every token: the groups before it win, the others lose
        z[:, :, 1] += np.float32(4) * np.arange(groups, dtype=np.float32)[::-1][None]
        z[:, :, 1] -= np.float32(2 * groups)
        z[:, top] = z[:, top - 1]
    else:
        z[:] = z[:, :1]
    steps = rng.integers(-40, 41, size=(T, groups, per)).astype(np.float32)
    z += steps * np.spacing(abs(z))
    z, bias = z.reshape(T, E), bias.reshape(E)
    want = chosen_by_groups(z, 2 * top, bias, groups, top)
    few, _ = ref.choose(z[:50], 2 * top, "sigmoid", bias, groups, top)
    assert np.array_equal(want[:50], few)
    got = choose(z, 2 * top, moe.Router("sigmoid", True, 1.0, groups, top), bias)
    wrong = np.nonzero((got != want).any(axis=1))[0]
    assert wrong.size == 0, (wrong.size, wrong[:5], got[wrong[:3]], want[wrong[:3]])


LOWEST = np.float32(-3.4028234663852886e38)


@pytest.mark.parametrize("E,groups", [(64, 4), (60, 4), (256, 8), (250, 5), (48, 3)])
def test_groups_barred_by_the_lowest_bias(E, groups):
    """A bias of float32's lowest value bars experts without removing them: two
    such keys sum to -infinity, but their group takes part behind the others (as
    one whose keys are all -infinity does, the lower of equal groups first)."""
    rng = np.random.default_rng(E)
    T, per = 60, E // groups
    for top in range(1, groups + 1):
        for barred in ("all", "groups", "most", "one group", "half"):
            bias = (rng.normal(size=E) * 0.1).astype(np.float32)
            bias = bias.reshape(groups, per)
            if barred == "all":
                bias[:] = LOWEST
            elif barred == "groups":  # all but one group
                bias[np.arange(groups) != groups // 2] = LOWEST
            elif barred == "most":    # one expert left in each, none in the first
                bias[:, 1:] = LOWEST
                bias[0] = LOWEST
            elif barred == "one group":
                bias[0] = LOWEST
            else:
                bias[rng.random((groups, per)) < 0.5] = LOWEST
            bias = bias.reshape(E)
            z = rng.normal(size=(T, E)).astype(np.float32)
            zg = z.reshape(T, groups, per)
            zg[10:20, 0] = -np.inf          # a group without any key, before barred ones
            zg[20:30, 1:] = -np.inf         # only the first group has keys
            zg[30:35, : groups - 1] = -np.inf
            zg[35:40, :, : per - 1] = -np.inf  # one key a group
            for k in (3, 8):
                say(f"[barred] E={E} groups={groups} top={top} {barred} k={k}")
                want, flagged = ref.choose(z, k, "sigmoid", bias, groups, top)
                assert not flagged
                got = choose(z, k, moe.Router("sigmoid", True, 1.0, groups, top), bias)
                assert np.array_equal(got, want), (np.nonzero((got != want).any(axis=1))[0],)


def test_groups_next_to_the_ends_of_float32():
    """Scores that overflow to either infinity, or just do not."""
    rng = np.random.default_rng(3)
    T, E, groups = 200, 64, 4
    for big in (1.7014117e38, 1.7014118e38, 1.7014120e38, 3.0e38, 3.4e38):
        for sign in (1.0, -1.0):
            bias = np.full((groups, 16), -LOWEST * np.float32(-0.5), np.float32)
            bias += (rng.integers(-3, 4, size=bias.shape) * 2.0 ** 103).astype(np.float32)
            bias[:, :2] = np.float32(sign * big)
            if sign < 0:
                bias[:, 2:] = LOWEST
            bias[1, 0] = np.nextafter(bias[1, 0], np.float32(0))
            bias[2, 1] = np.nextafter(bias[2, 1], np.float32(0))
            bias = bias.reshape(E)
            z = rng.normal(size=(T, E)).astype(np.float32)
            for top in (1, 2, 3):
                want, flagged = ref.choose(z, 6, "sigmoid", bias, groups, top)
                assert not flagged
                got = choose(z, 6, moe.Router("sigmoid", True, 1.0, groups, top), bias)
                assert np.array_equal(got, want), (big, sign, top)
