"""The router, its gradient and the balance loss on the GPU against the 64-bit
formulas: ids and counts exactly, floats to a count of their roundings.

Tolerances, in ULP = 2^-24 (half a step of float32, relative): an exponential
is off by 2 roundings of its own and by its argument's rounding, |difference
of logits| of them; a sum of n positive terms by at most as many roundings as
it has steps (a wave's over E experts: E / 64 in a lane and 6 across lanes);
each product or quotient adds one. Written out where they are used."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe
import router_ref as ref
from router_ref import ULP

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# half a step of the output, relative, and half the smallest step
STEP = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134),
        "f16": (2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


def say(msg):
    print(msg, flush=True)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def logits(rng, T, E, dtype, spread=1.0, ties=False):
    z = rng.normal(size=(T, E)) * spread
    if ties:
        z = np.round(z * 2) / 2
    t = torch.from_numpy(z.astype(np.float32)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


def run_route(z_d, k, router, bias=None, mask=None):
    T = z_d.shape[0]
    # a row before and behind, which must stay as they are
    ids = torch.full((T + 2, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, k), -77.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.route(z_d, k, router, ids[1:T + 1], w[1:T + 1], bias=bias, token_mask=mask, err=err)
    torch.cuda.synchronize()
    assert (ids[0] == -77).all() and (ids[-1] == -77).all()
    assert (w[0] == -77).all() and (w[-1] == -77).all()
    return ids[1:T + 1].cpu().numpy(), w[1:T + 1].cpu().numpy().astype(np.float64), int(err.item())


def weight_bound(z, ids, want, E):
    """Exponent argument (spread), its exponential (2), 1 + e, the quotients
    (3), the sum (k, or E / 64 + 6 over all), the scale; and the smallest
    floats, below which a weight is flushed or subnormal."""
    fin = z[np.isfinite(z)]
    spread = float(fin.max() - fin.min()) + abs(fin).max() if fin.size else 0.0
    spread = min(spread, 110.0)  # an exponential below e^-104 is 0
    n = max(ids.shape[1], E / 64 + 6)
    return abs(want) * (2 * spread + n + 12) * ULP + 2.0 ** -120


# (T, E, k, dtype, scoring, renorm, bias, groups, top_groups, ties)
ROUTES = [
    (1, 1, 1, "f32", "softmax", True, False, 1, 1, False),
    (1, 256, 8, "bf16", "sigmoid", True, True, 8, 4, False),
    (3, 7, 16, "f32", "softmax", True, False, 1, 1, False),     # more slots than experts
    (5, 63, 5, "f16", "softmax", False, False, 1, 1, False),
    (64, 384, 6, "f32", "softmax", True, False, 1, 1, False),
    (65, 65, 3, "bf16", "softmax", True, False, 1, 1, True),
    (257, 512, 8, "f32", "sigmoid", False, False, 1, 1, True),
    (130, 1024, 16, "f32", "softmax", False, False, 1, 1, False),
    (130, 1000, 7, "f16", "sigmoid", True, True, 1, 1, True),
    (100, 1024, 16, "bf16", "sigmoid", True, True, 64, 3, False),
    (100, 160, 8, "f32", "sigmoid", True, True, 8, 3, True),
    (100, 24, 4, "f32", "sigmoid", True, False, 24, 5, False),  # groups of one
    (100, 36, 6, "f32", "sigmoid", False, True, 3, 2, True),
    (1500, 256, 8, "f32", "sigmoid", True, True, 8, 4, False),
    (33, 128, 2, "f16", "softmax", True, False, 1, 1, True),
]


@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route(case):
    T, E, k, dt, scoring, renorm, bias, groups, top, ties = ROUTES[case]
    say(f"[route] {ROUTES[case]}")
    rng = np.random.default_rng(100 + case)
    z_d, z = logits(rng, T, E, dt, 1.5, ties)
    b = (rng.normal(size=E) * 0.1).astype(np.float32) if bias else None
    mask = rng.random(T) < 0.8 if case % 2 else None
    router = moe.Router(scoring, renorm, 2.5, groups, top)
    ids, w, err = run_route(z_d, k, router, None if b is None else dev(b),
                            None if mask is None else dev(mask))
    want, flagged = ref.choose(z, k, scoring, b, groups, top, mask)
    assert np.array_equal(ids, want)
    assert err == 0 and not flagged
    ww = ref.weights(z, want, scoring, renorm, 2.5)
    assert (abs(w - ww) <= weight_bound(z, ids, ww, E)).all()


LOW = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38, "f16": -65504.0}


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_experts(dt, scoring, renorm, groups):
    """-infinity is never chosen, the type's lowest value is an ordinary logit,
    a NaN or +infinity drops its token and says so, a masked token's logits are
    not looked at."""
    if scoring == "softmax" and groups > 1:
        groups = 1
    rng = np.random.default_rng(7)
    T, E, k = 40, 32, 5
    z_d, _ = logits(rng, T, E, dt)
    z_d[0] = -np.inf                 # nothing left
    z_d[1, 3:] = -np.inf             # fewer experts than slots
    z_d[2] = LOW[dt]                 # all lowest: ties by the lower id
    z_d[3, 4:] = LOW[dt]
    z_d[4, 2:30] = -np.inf
    z_d[5, 9] = float("nan")
    z_d[6, 31] = np.inf
    z_d[7] = float("nan")            # masked below
    z_d[8, 1] = np.inf               # masked below
    z_d[9] = 0.0
    z_d[9, ::2] = -0.0               # equal to +0
    z_d[10, 8:] = -np.inf            # whole groups gone
    z_d[11] = -60.0                  # sigmoids far below 1
    z_d[11, 5] = -61.0
    z = z_d.double().cpu().numpy()
    mask = np.ones(T, bool)
    mask[[7, 8, 20]] = False
    router = moe.Router(scoring, renorm, 1.0, groups, max(1, groups // 2))
    ids, w, err = run_route(z_d, k, router, None, dev(mask))
    want, flagged = ref.choose(z, k, scoring, None, groups, max(1, groups // 2), mask)
    assert flagged and err == moe.ERRBIT_BAD_LOGIT
    assert np.array_equal(ids, want)
    assert np.isfinite(w).all()
    zf = np.where(np.isfinite(z), z, 0.0)
    zf[zf <= LOW[dt]] = 0.0
    # rows 5 and 6 hold no weight: their ids are all -1
    ww = ref.weights(np.where(np.isnan(z) | (z == np.inf), 0.0, z), want, scoring, renorm, 1.0)
    assert (abs(w - ww) <= weight_bound(zf, ids, ww, E)).all()
    mask[[5, 6]] = False
    _, _, err = run_route(z_d, k, router, None, dev(mask))
    assert err == 0


def test_route_bad_bias():
    """A bias of -infinity bars its expert; one of NaN or +infinity is flagged."""
    rng = np.random.default_rng(8)
    z_d, z = logits(rng, 9, 40, "f32")
    b = np.zeros(40, np.float32)
    b[[0, 7, 39]] = -np.inf
    ids, _, err = run_route(z_d, 4, moe.Router("sigmoid"), dev(b))
    want, _ = ref.choose(z, 4, "sigmoid", b)
    assert err == 0 and np.array_equal(ids, want)
    b[3] = np.inf
    ids, w, err = run_route(z_d, 4, moe.Router("sigmoid"), dev(b))
    assert err == moe.ERRBIT_BAD_LOGIT and (ids == -1).all() and (w == 0).all()


def test_route_near_ties():
    """Scores a last bit apart: keys are the nearest floats of the sigmoid, so
    the choice among logits that differ by single steps is the formula's."""
    rng = np.random.default_rng(9)
    T, E, k = 400, 64, 8
    base = rng.normal(size=(T, 1)).astype(np.float32)
    step = rng.integers(-6, 7, size=(T, E)).astype(np.float32)
    z = base + step * np.spacing(np.abs(base))
    b = rng.integers(0, 2, size=E).astype(np.float32) * np.float32(2.0 ** -24)
    ids, _, err = run_route(dev(z), k, moe.Router("sigmoid"), dev(b))
    want, _ = ref.choose(z, k, "sigmoid", b)
    assert err == 0 and np.array_equal(ids, want)


def offsets_of(rng, T, S, first=0, last=None):
    last = T if last is None else last
    cuts = np.sort(rng.integers(first, last + 1, size=max(0, S - 1)))
    return np.concatenate([[first], cuts, [last]]).astype(np.int32)


def random_ids(rng, T, E, k):
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    ids[rng.random(T) < 0.1] = -1
    return ids


def run_balance(z_d, ids, scoring, S, off):
    T, E = z_d.shape
    k = ids.shape[1]
    need = moe.balance_workspace_bytes(T, E, k, S)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.full((S,), -7.0, device="cuda"),
           torch.full((S, E), -7, dtype=torch.int32, device="cuda"),
           torch.full((S,), -7, dtype=torch.int32, device="cuda"),
           torch.full((S, E), -7.0, device="cuda")]
    moe.balance_loss(z_d, ids, moe.Router(scoring), *out, workspace=ws[:need], err=err,
                     seq_offsets=off)
    torch.cuda.synchronize()
    assert (ws[need:] == 0x5A).all()
    return [o.cpu().numpy() for o in out], int(err.item())


# (T, E, k, dtype, scoring, S, first, tail)
BALANCES = [
    (0, 8, 2, "f32", "softmax", 1, 0, 0), (1, 1, 1, "f32", "softmax", 1, 0, 0),
    (31, 5, 2, "f16", "sigmoid", 1, 0, 0), (33, 64, 6, "bf16", "softmax", 5, 0, 0),
    (200, 384, 6, "f32", "sigmoid", 40, 3, 20), (129, 1024, 16, "f32", "softmax", 3, 0, 5),
    (2000, 130, 8, "bf16", "sigmoid", 7, 0, 300), (5000, 256, 8, "f32", "softmax", 300, 0, 0),
    (9001, 24, 3, "f16", "softmax", 2, 100, 0), (64, 16, 2, "f32", "softmax", 2000, 0, 0),
]


@pytest.mark.parametrize("case", range(len(BALANCES)))
def test_balance(case):
    T, E, k, dt, scoring, S, first, tail = BALANCES[case]
    say(f"[balance] {BALANCES[case]}")
    rng = np.random.default_rng(200 + case)
    z_d, z = logits(rng, T, E, dt, 1.5)
    ids = random_ids(rng, T, E, k)
    off = offsets_of(rng, T, S, first, T - tail)
    used = S > 1 or first or tail
    (loss, counts, tokens, mean), err = run_balance(z_d, dev(ids), scoring, S,
                                                    dev(off) if used else None)
    wl, wc, wt, wm = ref.balance(z, ids, scoring, off)
    assert err == 0
    assert np.array_equal(counts, wc) and np.array_equal(tokens, wt)
    # a share: argument (spread), exponential (2), 1 + e, sum over E, quotient;
    # then at most 16 + tile / 16 additions in floats, the rest in doubles
    spread = 0.0 if T == 0 else float(z.max() - z.min()) + abs(z).max()
    tile = max(32, T // 128 + 16)
    rel = (2 * spread + E / 64 + 6 + 12 + 16 + tile / 16) * ULP
    assert (abs(mean - wm) <= wm * rel + 1e-37).all()
    assert (abs(loss - wl) <= wl * (rel + 2 * ULP) + 1e-37).all()


def test_balance_unused_logits_and_extremes():
    """Logits of tokens without an expert or outside the sequences may be
    anything; -infinity and the lowest value are a share of 0; a row that has
    nothing else adds nothing; ids out of range are flagged."""
    rng = np.random.default_rng(11)
    T, E, k = 70, 40, 3
    for scoring in ("softmax", "sigmoid"):
        z_d, _ = logits(rng, T, E, "f32")
        ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
        ids[5] = -1
        z_d[5] = float("nan")
        z_d[:2] = float("nan")
        z_d[66:] = np.inf
        z_d[10, 3:] = -np.inf
        z_d[11, 1:] = LOW["f32"]
        z_d[12] = -np.inf
        z_d[13] = -300.0
        off = np.array([2, 20, 66], np.int32)
        z = z_d.double().cpu().numpy()
        keep = np.where(np.isnan(z) | (z == np.inf), 0.0, z)
        (loss, counts, tokens, mean), err = run_balance(z_d, dev(ids), scoring, 2, dev(off))
        wl, wc, wt, wm = ref.balance(keep, ids, scoring, off)
        assert err == 0
        assert np.array_equal(counts, wc) and np.array_equal(tokens, wt)
        # as above with a spread of at most 110 (beyond it an exponential is 0)
        assert (abs(mean - wm) <= wm * 300 * ULP + 1e-37).all()
        assert (abs(loss - wl) <= wl * 300 * ULP).all()
        ids[30, 1] = E
        ids[31, 0] = -2
        (_, counts, tokens, _), err = run_balance(z_d, dev(ids), scoring, 2, dev(off))
        _, wc, wt, _ = ref.balance(keep, ids, scoring, off)
        assert err == moe.ERRBIT_BAD_ID
        assert np.array_equal(counts, wc) and np.array_equal(tokens, wt)


def test_balance_flags_bad_offsets():
    rng = np.random.default_rng(12)
    z_d, _ = logits(rng, 50, 8, "f32")
    ids = dev(random_ids(rng, 50, 8, 2))
    for off in ([0, 30, 20, 50], [0, 10, 20, 51], [-1, 10, 20, 50], [0, 2 ** 31 - 1, -5, 50]):
        _, err = run_balance(z_d, ids, "softmax", 3, dev(np.array(off, np.int32)))
        assert err & moe.ERRBIT_BAD_SEQ, off


# (T, E, k, dtype, scoring, renorm, weights, S (0: no balance loss), first, tail)
GRADS = [
    (1, 1, 1, "f32", "softmax", True, True, 1, 0, 0),
    (1, 256, 8, "bf16", "sigmoid", True, True, 0, 0, 0),
    (5, 63, 5, "f16", "softmax", False, True, 0, 0, 0),
    (64, 384, 6, "f32", "softmax", True, True, 0, 0, 0),
    (64, 384, 6, "f32", "softmax", False, True, 3, 0, 0),
    (130, 1024, 16, "f32", "sigmoid", False, True, 4, 2, 9),
    (130, 1000, 7, "f16", "sigmoid", True, True, 1, 0, 0),
    (300, 160, 8, "bf16", "sigmoid", True, False, 30, 0, 17),
    (300, 24, 4, "f32", "softmax", True, False, 1, 0, 0),
    (1500, 256, 8, "f32", "softmax", True, True, 13, 0, 100),
]


def run_grad(z_d, ids, router, dw=None, balance=None):
    T, E = z_d.shape
    d = torch.full((T + 2, E), -77.0, dtype=z_d.dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.route_backward(z_d, ids, router, d[1:T + 1], d_weights=dw, balance=balance, err=err)
    torch.cuda.synchronize()
    assert (d[0] == -77).all() and (d[-1] == -77).all()
    return d[1:T + 1].double().cpu().numpy(), int(err.item())


def grad_bound(want, size, E, k, dt, spread):
    """Every absolute term of the sum (size) is a product of factors that are
    each off by a spread's rounding, an exponential, a sum over E or k and a few
    single roundings; then the output's own half step."""
    rel, least = STEP[dt]
    return (2 * min(spread, 110.0) + E / 64 + 6 + 2 * k + 24) * ULP * size + abs(want) * rel + \
        least + 1e-37


@pytest.mark.parametrize("case", range(len(GRADS)))
def test_gradient(case):
    T, E, k, dt, scoring, renorm, weights, S, first, tail = GRADS[case]
    say(f"[gradient] {GRADS[case]}")
    rng = np.random.default_rng(300 + case)
    z_d, z = logits(rng, T, E, dt, 1.5)
    ids = random_ids(rng, T, E, k)
    ids[0, 0] = 0
    if T > 2 and k > 1:
        ids[1, :2] = E // 2      # the same expert twice
        ids[2] = E - 1           # in all slots
    dw = rng.normal(size=(T, k)).astype(np.float32) if weights else None
    if dw is not None:
        dw[ids < 0] = np.nan     # never read
    off = offsets_of(rng, T, S, first, T - tail) if S else None
    dl = rng.normal(size=S).astype(np.float32) if S else None
    balance = None
    if S:
        _, counts, tokens, _ = ref.balance(z, ids, scoring, off)
        balance = (dev(dl), dev(counts.astype(np.int32)), dev(tokens.astype(np.int32)),
                   dev(off) if S > 1 else None)
    router = moe.Router(scoring, renorm, 2.5)
    got, err = run_grad(z_d, dev(ids), router, None if dw is None else dev(dw), balance)
    want, size = ref.gradient(z, ids, scoring, renorm, 2.5, dw, dl, off)
    assert err == 0
    spread = float(z.max() - z.min()) + abs(z).max()
    assert (abs(got - want) <= grad_bound(want, size, E, k, dt, spread)).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_extremes(scoring, renorm):
    """Masked experts have no gradient, tokens without an expert none at all
    whatever their logits hold, and scores far below 1 do not turn to NaN."""
    rng = np.random.default_rng(13)
    T, E, k = 30, 40, 3
    z_d, _ = logits(rng, T, E, "f32")
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[0] = -1
    z_d[0] = float("nan")
    z_d[1, 10:] = -np.inf
    ids[1] = [1, 2, 20]              # a chosen expert with a score of 0
    z_d[2, 5:] = -np.inf
    ids[2] = [10, 11, 12]            # only such
    z_d[3] = -200.0
    z_d[4] = 200.0
    z_d[5, 1:] = LOW["f32"]
    z_d[6] = -np.inf
    z = z_d.double().cpu().numpy()
    z = np.where(np.isnan(z), 0.0, z)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    off = np.array([0, T], np.int32)
    dl = np.array([0.7], np.float32)
    _, counts, tokens, _ = ref.balance(z, ids, scoring, off)
    got, err = run_grad(z_d, dev(ids), moe.Router(scoring, renorm, 1.0), dev(dw),
                        (dev(dl), dev(counts.astype(np.int32)), dev(tokens.astype(np.int32)),
                         None))
    want, size = ref.gradient(z, ids, scoring, renorm, 1.0, dw, dl, off)
    assert err == 0 and np.isfinite(got).all()
    assert (abs(got - want) <= grad_bound(want, size, E, k, "f32", 110.0)).all()


def test_gradient_bad_ids_and_empty():
    rng = np.random.default_rng(14)
    z_d, z = logits(rng, 20, 16, "f32")
    ids = random_ids(rng, 20, 16, 2)
    ids[3] = [16, 4]
    ids[4] = [-2, -1]
    dw = rng.normal(size=(20, 2)).astype(np.float32)
    got, err = run_grad(z_d, dev(ids), moe.Router(), dev(dw))
    want, size = ref.gradient(z, ids, "softmax", True, 1.0, dw)
    assert err == moe.ERRBIT_BAD_ID
    assert (abs(got - want) <= grad_bound(want, size, 16, 2, "f32", 12.0)).all()
    assert (got[4] == 0).all()
    got, err = run_grad(z_d[:0], dev(ids[:0]), moe.Router(), dev(dw[:0]))
    assert err == 0 and got.shape == (0, 16)


def test_gradient_against_differences():
    """A step along the GPU's gradient changes the 64-bit loss as it says:
    central differences with h = 1e-4 (off by about h^2 times third
    derivatives of size 1) against <gradient, direction>."""
    rng = np.random.default_rng(15)
    T, E, k = 50, 48, 6
    off = np.array([0, 11, 11, 44], np.int32)
    for scoring in ("softmax", "sigmoid"):
        z_d, z = logits(rng, T, E, "f32")
        ids = ref.choose(z, k, scoring)[0].astype(np.int32)
        dw = rng.normal(size=(T, k)).astype(np.float32)
        dl = rng.normal(size=3).astype(np.float32)
        _, counts, tokens, _ = ref.balance(z, ids, scoring, off)
        got, _ = run_grad(z_d, dev(ids), moe.Router(scoring), dev(dw),
                          (dev(dl), dev(counts.astype(np.int32)), dev(tokens.astype(np.int32)),
                           dev(off)))

        def value(z):
            return ((ref.weights(z, ids, scoring, True, 1.0) * dw).sum()
                    + (ref.balance(z, ids, scoring, off)[0] * dl).sum())

        for _ in range(4):
            v = rng.normal(size=z.shape)
            h = 1e-4
            slope = (value(z + h * v) - value(z - h * v)) / (2 * h)
            # T * E elements of the float gradient, each off by some ULP of its
            # terms (at most 2.5 in size here), and the differences' own error
            assert abs(slope - (got * v).sum()) < 1e-5
