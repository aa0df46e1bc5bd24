"""Calls at borders: group scores whose keys are much larger than their sum,
or sum to an infinity; shares of logits as far out as their type goes; one
workspace for batches of all sizes; the products of a slice of the experts."""
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


def far_rows(E, dtype):
    """Logits near the ends of the type, one kind a row, all finite or masked."""
    info = torch.finfo(dtype)
    rng = np.random.default_rng(17)
    z = torch.from_numpy(rng.normal(size=(64, E)).astype(np.float32)).to(dtype)
    z[0] = info.min                      # all lowest: even shares
    z[1] = info.min
    z[1, 3] = -1.0                       # one share
    z[2] = info.min
    z[2, 5:] = -float("inf")             # five shares
    z[3] = info.max
    z[4, 7] = info.max                   # one share, or (sigmoid) about even ones
    z[5] = info.max * 0.75
    z[5, 2:] = info.max * 0.5            # two shares
    z[6] = info.min * 0.75
    z[6, 4:] = info.min                  # four
    z[7] = info.min * 0.25
    z[7, 9] = info.min * 0.125
    z[8] = info.max * 0.71               # about where log2(e) times it passes the end
    z[9] = info.min * 0.71
    z[10] = info.max * 0.68
    z[11] = info.min * 0.68
    z[12, :] = info.min
    z[12, 6] = info.max
    # 13: ordinary; behind it a step or some of the type apart, from 4 on up, of
    # both signs (1.44 times such a logit is rounded by much more than 1)
    for i in range(14, 64):
        base = torch.tensor(3.0 * 2.0 ** (i - 13) * (-1) ** i).clamp(info.min / 2, info.max / 2)
        base = base.to(dtype)
        step = 2.0 ** torch.frexp(base.double().abs())[1] * info.eps / 2
        near = torch.from_numpy(rng.integers(-3, 4, size=E))
        z[i] = (base.double() + near * step).to(dtype)
    return z


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [40, 64, 600])
def test_shares_of_far_logits(dtype, scoring, E):
    """The balance loss and the gradient where every logit of a token is finite
    but as far out as its type goes."""
    say(f"[far] {dtype} {scoring} E={E}")
    z_d = far_rows(E, dtype).cuda()
    z = z_d.double().cpu().numpy()
    T, k = z.shape[0], 3
    rng = np.random.default_rng(18)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[:, 0] = 3
    i32 = dict(dtype=torch.int32, device="cuda")
    ids_d = torch.from_numpy(ids).cuda()
    err = torch.zeros(1, **i32)
    off = np.arange(T + 1)               # a sequence per row: its shares are its means
    off_d = torch.arange(T + 1, **i32)
    loss, mean = torch.full((T,), -7.0, device="cuda"), torch.full((T, E), -7.0, device="cuda")
    counts, tokens = torch.full((T, E), -7, **i32), torch.full((T,), -7, **i32)
    ws = torch.empty(moe.balance_workspace_bytes(T, E, k, T), dtype=torch.uint8, device="cuda")
    moe.balance_loss(z_d, ids_d, moe.Router(scoring), loss, counts, tokens, mean, workspace=ws,
                     seq_offsets=off_d, err=err)
    torch.cuda.synchronize()
    wl, wc, wt, wm = ref.balance(z, ids, scoring, off)
    assert int(err.item()) == 0
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(tokens.cpu().numpy(), wt)
    # a share: its exponential and argument (an exponent of at most 110, beyond
    # it is 0), the sum over E and three single roundings
    rel = (2 * 110 + E / 16 + 8) * ref.ULP
    assert (abs(mean.double().cpu().numpy() - wm) <= wm * rel + 1e-37).all()
    # a share below 2^-126 may be 0: each of the k pairs of the one token adds E / k
    # times its expert's share, so a loss is off by at most E * 2^-126 for that
    assert (abs(loss.double().cpu().numpy() - wl) <= wl * (rel + 2 * ref.ULP) +
            E * 2.0 ** -126).all()

    dw = rng.normal(size=(T, k)).astype(np.float32)
    dl = rng.normal(size=T).astype(np.float32)
    step, least = {torch.float32: (0.0, 0.0), torch.bfloat16: (2.0 ** -8, 0.0),
                   torch.float16: (2.0 ** -11, 2.0 ** -25)}[dtype]
    # and p (u - sum p u) with every p off by at most 2^-126: by 2^-126 of |u| and of
    # sum |u| twice (|sum p u| <= sum |u|), where sum |u| <= |d_loss| E / k * (k + k)
    # from the counts and k T' / E, and sum |d_weights| from the raw weights
    flushed = 3 * 2.0 ** -126 * (2 * E * abs(dl) + abs(dw).sum(axis=1)).astype(np.float64)[:, None]
    for renorm in (True, False):
        dz = torch.full((T, E), -7.0, dtype=dtype, device="cuda")
        moe.route_backward(z_d, ids_d, moe.Router(scoring, renorm), dz,
                           d_weights=torch.from_numpy(dw).cuda(),
                           balance=(torch.from_numpy(dl).cuda(), counts, tokens, off_d), err=err)
        torch.cuda.synchronize()
        want, size = ref.gradient(z, ids, scoring, renorm, 1.0, dw, dl, off)
        got = dz.double().cpu().numpy()
        assert int(err.item()) == 0 and np.isfinite(got).all()
        # as above, the quotients and sums over k, then the output's half step
        bound = (rel + (2 * k + 16) * ref.ULP) * size * (1 + step) + step * abs(want) + least + flushed
        assert (abs(got - want) <= bound).all()


@pytest.mark.parametrize("most,T", [(2049, 2048), (2049, 33), (16385, 16384), (16385, 4097)])
def test_balance_workspace_of_a_larger_batch(most, T):
    """One workspace, made for the largest batch: smaller ones fit, and give what
    they give in one of their own."""
    E, k, S = 48, 4, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    z = torch.randn(T, E, device="cuda", generator=g)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    off = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for size in (moe.balance_workspace_bytes(most, E, k, S), moe.balance_workspace_bytes(T, E, k, S)):
        ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        out = [torch.full((S,), -7.0, device="cuda"), torch.full((S, E), -7, **i32),
               torch.full((S,), -7, **i32), torch.full((S, E), -7.0, device="cuda")]
        moe.balance_loss(z, ids, moe.Router(), *out, workspace=ws[:size], seq_offsets=off, err=err)
        torch.cuda.synchronize()
        assert bool((ws[size:] == 0x5A).all()) and int(err.item()) == 0
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    _, wc, wt, _ = ref.balance(z.double().cpu().numpy(), ids.cpu().numpy(), "softmax",
                               off.cpu().numpy())
    assert (got[0][1].cpu().numpy() == wc).all() and (got[0][2].cpu().numpy() == wt).all()


@pytest.mark.parametrize("share", [150, 25, 4, 1])
def test_product_of_a_slice_with_its_share_of_the_rows(share):
    """The experts [a, b) of a layout with T * k the whole layout's rows, theirs,
    or fewer: the same rows are written, each within its roundings."""
    from test_experts_gpu import i32, layout, weights
    rng = np.random.default_rng(31)
    counts, H, N = [50, 9, 0, 12, 4, 75], 192, 40
    off = layout(counts, 1, 0)
    x = torch.from_numpy(rng.normal(size=(150, H)).astype(np.float32)).to(torch.bfloat16)
    q, s = weights(rng, "mxfp4", 6, N, H)
    out = torch.full((150, N), -77.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.expert_product("mxfp4", x.cuda(), i32(counts)[1:5], i32(off)[1:6], share, 1,
                       torch.from_numpy(q[1:5]).cuda(), torch.from_numpy(s[1:5]).cuda(), out, err=err)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert int(err.item()) == 0
    assert (got[:50] == -77).all() and (got[75:] == -77).all()
    for e in range(1, 5):
        at = slice(int(off[e]), int(off[e + 1]))
        w, xd = ref.weight_values("mxfp4", q[e], s[e]), x[at].double().numpy()
        want, size = xd @ w.T, abs(xd) @ abs(w.T)
        # counted as in test_experts_gpu.py
        bound = (H / 32 * 8 + 8) * ref.ULP * size + 2.0 ** -8 * abs(want)
        assert (abs(got[at] - want) <= bound).all()
