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
