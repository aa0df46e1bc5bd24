"""The expert products with 4-bit weights on the GPU against the 64-bit
formula.

Tolerance: a weight's value is exact in bf16 and a product of two bf16 values
in float32; the sum over H runs through MFMA instructions of 32 products each,
taken as at most 8 roundings per instruction, so y is off by at most
(H / 32 * 8 + 8) * 2^-24 * sum |w x| (8 for the joining of partial sums, factor
and conversion), and the bf16 output by half a step, 2^-8 of the value. SwiGLU
passes an error of the gate on with a slope of at most 1.1."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe
import router_ref as ref
from router_ref import ULP

pytestmark = pytest.mark.gpu
GROUP = {"mxfp4": 32, "nvfp4": 16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


def say(msg):
    print(msg, flush=True)


def layout(counts, align, block):
    counts = np.asarray(counts, np.int64)
    if block:
        return np.arange(len(counts) + 1) * block
    runs = -(-counts // align) * align
    return np.concatenate([[0], np.cumsum(runs)])


def rows_in_use(counts, off, cap):
    out = np.full(cap, -1, np.int64)
    for e, n in enumerate(counts):
        a = int(off[e])
        b = min(a + int(min(n, off[e + 1] - off[e])), cap)
        out[a:b] = e
    return out


def weights(rng, fmt, E, N, H):
    q = rng.integers(0, 256, size=(E, N, H // 2)).astype(np.uint8)
    lo, hi = (118, 126) if fmt == "mxfp4" else (8, 56)
    s = rng.integers(lo, hi, size=(E, N, H // GROUP[fmt])).astype(np.uint8)
    if fmt == "nvfp4":
        s |= (rng.random(s.shape) < 0.1).astype(np.uint8) << 7  # a scale may be negative
    return q, s


def run(fmt, rows, counts, off, T, k, q, s, act=None, factor=None, cap=None):
    """rows: bf16 tensor [cap, H] on the GPU. Returns out with a row before and
    behind, those two checked to be left alone, and the error word."""
    cap = rows.shape[0]
    N = q.shape[1] // 2 if act == "swiglu" else q.shape[1]
    out = torch.full(((cap + 2) * N + 64,), -77.0, dtype=torch.bfloat16, device="cuda")
    skip = -(-N // 8) * 8  # 16-byte alignment
    view = out[skip:skip + cap * N].view(cap, N)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.expert_product(fmt, rows, counts, off, T, k, q, s, view, act=act, factor=factor, err=err)
    torch.cuda.synchronize()
    assert (out[:skip] == -77).all() and (out[skip + cap * N:] == -77).all()
    return view, int(err.item())


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def check(fmt, counts, H, N, act, factor, align=1, block=0, cap=None, T=None, k=1, seed=0):
    rng = np.random.default_rng(seed)
    E = len(counts)
    off = layout(counts, align, block)
    full = max(int(off[-1]), 1)
    cap = full if cap is None else cap
    total = int(np.sum(counts))
    T = max(1, -(-total // k)) if T is None else T
    use = rows_in_use(counts, off, cap)
    x = torch.from_numpy(rng.normal(size=(cap, H)).astype(np.float32)).to(torch.bfloat16)
    x[torch.from_numpy(use < 0)] = float("nan")  # rows not in use are never taken in
    q, s = weights(rng, fmt, E, N, H)
    f = rng.uniform(-2, 2, size=E).astype(np.float32) if factor else None
    got, err = run(fmt, x.cuda(), i32(counts), i32(off), T, k, torch.from_numpy(q).cuda(),
                   torch.from_numpy(s).cuda(), act, None if f is None else torch.from_numpy(f).cuda())
    got = got.double().cpu().numpy()
    assert (got[use < 0] == -77).all(), "a row that is not in use was written"
    full_rows = rows_in_use(counts, off, max(full, cap))
    assert err == (moe.ERRBIT_EXPERT_CAP if (full_rows >= 0).sum() > (use >= 0).sum() else 0)
    xd = x.double().numpy()
    gamma = (H / 32 * 8 + 8) * ULP
    for e in range(E):
        at = np.nonzero(use == e)[0]
        if at.size == 0:
            continue
        w = ref.weight_values(fmt, q[e], s[e])
        c = 1.0 if f is None else float(f[e])
        y, size = xd[at] @ w.T * c, abs(xd[at]) @ abs(w.T) * abs(c)
        tol = gamma * size
        if act == "swiglu":
            g, u = y[:, :N // 2], y[:, N // 2:]
            silu = g * ref.sigmoid(g)
            y = silu * u
            tol = 1.1 * tol[:, :N // 2] * (abs(u) + tol[:, N // 2:]) + \
                (abs(silu)) * tol[:, N // 2:] + 16 * ULP * abs(y) * (1 + abs(g))
        bad = abs(got[at] - y) > tol + 2.0 ** -8 * abs(y) + 1e-37
        assert not bad.any(), (e, np.argwhere(bad)[:3], got[at][bad][:3], y[bad][:3])


SHAPES = [
    # counts, H, N, act, factor, align, block
    ([1], 32, 1, None, False, 1, 0),
    ([0, 0, 1, 0], 64, 17, None, False, 1, 0),
    ([1, 1, 1, 1, 1, 1], 512, 64, "swiglu", False, 1, 0),
    ([3, 0, 16, 17, 1, 0, 15], 96, 33, None, True, 1, 0),
    ([2, 5, 0, 9], 160, 48, "swiglu", True, 16, 0),
    ([33, 1, 64, 65], 416, 40, "swiglu", False, 1, 0),
    ([130, 7, 0], 1056, 100, None, False, 1, 0),
    ([5, 12, 0, 3], 2048, 130, None, True, 1, 16),
    ([20, 40, 0, 3], 544, 66, "swiglu", False, 1, 16),   # blocks fuller than they are
    ([300], 256, 70, None, False, 128, 0),
    ([8] * 48, 5120, 96, "swiglu", True, 1, 0),
    ([1] * 3 + [0] * 1018 + [2] * 3, 128, 32, None, False, 1, 0),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_product(fmt, case):
    say(f"[product] {fmt} {SHAPES[case]}"[:150])
    counts, H, N, act, factor, align, block = SHAPES[case]
    check(fmt, counts, H, N, act, factor, align, block, seed=400 + case)


@pytest.mark.parametrize("seed", range(24))
def test_product_random_shapes(seed):
    rng = np.random.default_rng(4000 + seed)
    E = int(rng.integers(1, 40))
    most = int(rng.choice([1, 3, 20, 90]))
    counts = rng.integers(0, most + 1, size=E) * (rng.random(E) < 0.7)
    act = rng.choice([None, "swiglu"])
    N = int(rng.integers(1, 200))
    align = int(rng.choice([1, 1, 16, 128]))
    block = int(rng.integers(1, most + 2)) if align == 1 and rng.random() < 0.3 else 0
    H = 32 * int(rng.integers(1, 40))
    say(f"[product random] seed {seed} E={E} most={most} H={H} N={N} act={act} align={align} "
        f"block={block}")
    check(str(rng.choice(["mxfp4", "nvfp4"])), counts, H, N + N % 2 if act else N, act,
          bool(rng.random() < 0.5), align, block, seed=seed,
          k=int(rng.integers(1, 9)))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_small_buffer(fmt):
    """Rows the buffer does not hold are skipped and flagged."""
    for cap in (1, 5, 30, 39):
        check(fmt, [20, 0, 20], 64, 24, None, False, cap=cap, seed=cap)


def test_product_more_rows_than_said():
    """T * k below the rows in use costs time, not rows."""
    check("mxfp4", [40, 3, 0, 70], 128, 48, "swiglu", False, T=1, k=1, seed=5)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_exact_sums(fmt):
    """Every code, with small whole inputs: all sums are exact in float32, so
    the output is the nearest bf16 of the exact sum and nothing else."""
    rng = np.random.default_rng(21)
    H, N, counts = 480, 200, [1, 7, 0, 18]
    off = layout(counts, 1, 0)
    x = rng.integers(-3, 4, size=(26, H)).astype(np.float32)
    q = rng.integers(0, 256, size=(4, N, H // 2)).astype(np.uint8)
    if fmt == "mxfp4":
        s = rng.integers(126, 129, size=(4, N, H // 32)).astype(np.uint8)
    else:
        s = rng.integers(40, 72, size=(4, N, H // 16)).astype(np.uint8)
    got, err = run(fmt, torch.from_numpy(x).to(torch.bfloat16).cuda(), i32(counts), i32(off), 26,
                   1, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    use = rows_in_use(counts, off, 26)
    want = np.stack([ref.weight_values(fmt, q[e], s[e]) @ x[r].astype(np.float64)
                     for r, e in enumerate(use)])
    assert err == 0
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_every_code_and_scale():
    """One-hot inputs read every weight's value: all 16 codes under every scale
    byte of both formats, exactly (bf16 holds them; NaN scales give NaN)."""
    for fmt in ("mxfp4", "nvfp4"):
        blk = GROUP[fmt]
        H, N = 32, 256
        q = np.zeros((1, N, H // 2), np.uint8)
        q[:] = np.arange(16)[None, None, :] | (np.arange(16)[::-1][None, None, :] << 4)
        s = np.repeat(np.arange(256, dtype=np.uint8)[None, :, None], H // blk, axis=2)
        x = torch.eye(H).to(torch.bfloat16)
        # inputs are 0 elsewhere: 0 * infinity does not occur for values that
        # bf16 holds, so scales whose products pass its range are left out
        got, err = run(fmt, x.cuda(), i32([H]), i32([0, H]), H, 1, torch.from_numpy(q).cuda(),
                       torch.from_numpy(s).cuda())
        want = ref.weight_values(fmt, q[0], s[0]).T
        got = got.double().cpu().numpy()
        fits = np.abs(want).max(axis=0) <= 3.38e38
        nan = np.isnan(want).all(axis=0)
        assert err == 0 and fits.sum() >= 250
        assert np.array_equal(got[:, fits], want[:, fits]), fmt
        assert np.isnan(got[:, nan]).all(), fmt


def test_product_of_a_slice_of_the_experts():
    """The experts [a, b) of a layout by their slice of counts and offsets: the
    other experts' rows stay as they are."""
    rng = np.random.default_rng(23)
    counts = [4, 9, 0, 21, 3, 8]
    off = layout(counts, 1, 0)
    H, N = 192, 40
    x = torch.from_numpy(rng.normal(size=(45, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    q, s = (torch.from_numpy(v).cuda() for v in weights(rng, "mxfp4", 6, N, H))
    whole, _ = run("mxfp4", x, i32(counts), i32(off), 45, 1, q, s)
    part, err = run("mxfp4", x, i32(counts)[2:5], i32(off)[2:6], 45, 1, q[2:5], s[2:5])
    assert err == 0
    assert torch.equal(part[13:37], whole[13:37])
    assert (part[:13] == -77).all() and (part[37:] == -77).all()


def test_product_with_wild_counts():
    """Counts and offsets of any value: nothing outside the buffer is touched."""
    rng = np.random.default_rng(24)
    x = torch.from_numpy(rng.normal(size=(20, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    q, s = (torch.from_numpy(v).cuda() for v in weights(rng, "nvfp4", 3, 16, 64))
    for counts, off in (([-5, 100, 3], [0, 5, 9, 20]), ([5, 5, 5], [-3, 30, 10, 40]),
                        ([2, 2 ** 31 - 1, 1], [0, 2, 2 ** 31 - 1, 4])):
        run("nvfp4", x, i32(counts), i32(off), 20, 1, q, s)
