"""The products in 8-bit integers on the GPU against the formula.

Without an activation the result is determined to the bit: the sum is exact, and
rounded once to float32, once by each scale and once to bf16. SwiGLU is compared
in 64 bits: gate and up are off by 3 * 2^-24 of themselves each (a slope of at
most 1.1 passes the gate's on), the exponential, sum, quotient and products by at
most 10 more, and bf16 by half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


def say(msg):
    print(msg, flush=True)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def layout(counts, align, block):
    counts = np.asarray(counts, np.int64)
    if block:
        return np.arange(len(counts) + 1) * block
    return np.concatenate([[0], np.cumsum(-(-counts // align) * align)])


def check(q, xs, w, ws, act, got):
    """Rows q of one expert; everything on the GPU, the sums in 64-bit floats (exact)."""
    y = q.to(F64) @ w.to(F64).t().contiguous()
    assert float(y.abs().max()) < 2 ** 31
    f = y.to(torch.float32) * xs[:, None] * ws
    if act is None:
        assert torch.equal(got, f.to(torch.bfloat16))
        return
    y = y * xs.to(F64)[:, None] * ws.to(F64)
    n = y.shape[1] // 2
    gate, up = y[:, :n], y[:, n:]
    want = gate * torch.sigmoid(gate) * up
    bound = ULP * (3.3 * (gate * up).abs() + 13 * want.abs()) + 2.0 ** -8 * want.abs() + 1e-38
    off = (got.to(F64) - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def run(q, xs, w, ws, act, counts=None, off=None, T=None, k=1, cap=None):
    """The call into rows with guards before and behind; returns out and the error word."""
    cap = q.shape[0] if cap is None else cap
    N = w.shape[1]
    wide = N // 2 if act else N
    room = torch.full((16 + cap * wide + 64,), 0x5A5A, dtype=torch.int16, device="cuda")
    out = room[16:16 + cap * wide].view(cap, wide)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    moe.int8_product(q[:cap], xs[:cap], w, ws, out, act=act, T=T, k=k, err=err,
                     expert_counts=None if counts is None else torch.tensor(counts, **i32),
                     expert_offsets=None if off is None else torch.tensor(off, **i32))
    torch.cuda.synchronize()
    assert bool((room[:16] == 0x5A5A).all()) and bool((room[16 + cap * wide:] == 0x5A5A).all())
    return out, int(err.item())


def inputs(seed, rows, E, N, K):
    g = gen(seed)
    q, w = codes(g, rows, K), codes(g, E, N, K)
    xs = torch.exp(torch.randn(rows, generator=g, device="cuda")) / 64
    ws = torch.exp(torch.randn(E, N, generator=g, device="cuda")) / (64 * K ** 0.5)
    return q, xs, w, ws


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 100, 128, 129, 255, 256,
                                  257, 300, 520, 1000])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_plain_rows(rows, act):
    for N, K in [(2, 16), (34, 144), (256, 128), (130, 1040), (1000, 5120), (510, 2064),
                 (4096, 7168)]:
        if rows * N * K > 1 << 31:
            continue
        say(f"plain rows={rows} N={N} K={K} act={act}")
        q, xs, w, ws = inputs(rows * 7919 + N + K, rows, 1, N, K)
        out, err = run(q, xs, w, ws, act)
        assert err == 0
        check(q, xs, w[0], ws[0], act, out.view(torch.bfloat16))


@pytest.mark.parametrize("N", [1, 3, 15, 17, 31, 33, 127, 129, 255, 257])
@pytest.mark.parametrize("rows", [5, 40, 200, 2000])
def test_odd_columns(N, rows):
    for K in (16, 272, 400):
        q, xs, w, ws = inputs(N * 31 + rows + K, rows, 1, N, K)
        out, err = run(q, xs, w, ws, None)
        assert err == 0
        check(q, xs, w[0], ws[0], None, out.view(torch.bfloat16))


@pytest.mark.parametrize("N", [2050, 2054, 2060, 2064])  # with SwiGLU half as many columns
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("rows", [150, 700, 2100, 4099])
def test_rows_of_out_at_any_address(rows, act, N):
    q, xs, w, ws = inputs(rows + N, rows, 1, N, 528)
    out, err = run(q, xs, w, ws, act)
    assert err == 0
    check(q, xs, w[0], ws[0], act, out.view(torch.bfloat16))


def check_experts(q, xs, w, ws, act, counts, off, out):
    cap = out.shape[0]
    used = torch.zeros(cap, dtype=torch.bool, device="cuda")
    for e, n in enumerate(counts):
        a = int(off[e])
        b = min(a + int(min(n, off[e + 1] - off[e])), cap)
        if b > a:
            used[a:b] = True
            check(q[a:b], xs[a:b], w[e], ws[e], act, out[a:b].view(torch.bfloat16))
    assert bool((out[~used] == 0x5A5A).all())  # the other rows are left as they were


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("shape", ["runs", "padded", "blocks"])
@pytest.mark.parametrize("mean", [0.3, 2, 9, 20, 50, 120, 400])
def test_experts(mean, shape, act):
    rng = np.random.default_rng(int(mean * 10) + len(shape) + (act is not None))
    for E, N, K in [(1, 96, 208), (5, 66, 1024), (64, 64, 128), (130, 32, 64), (9, 520, 640)]:
        counts = rng.poisson(mean * np.exp(rng.normal(0, 0.7, E)))
        counts[rng.integers(E)] = 0
        if E > 2:
            counts[0], counts[1] = int(mean * 3) + 1, 1
        align = 48 if shape == "padded" else 1
        block = int(counts.max()) + 3 if shape == "blocks" else 0
        off = layout(counts, align, block)
        cap = int(off[-1]) + 5
        pairs = max(1, int(counts.sum()))
        say(f"experts mean={mean} {shape} act={act} E={E} N={N} K={K} rows={counts.sum()}")
        q, xs, w, ws = inputs(E + N + K, cap, E, N, K)
        out, err = run(q, xs, w, ws, act, counts, off, pairs, 1)
        assert err == 0
        check_experts(q, xs, w, ws, act, counts, off, out)


@pytest.mark.parametrize("T", [1, 3, 40, 700, 5000])
def test_launch_laid_out_for_another_number_of_rows(T):
    """Fewer or more rows than T * k: all rows in use are made."""
    counts = np.array([3, 0, 150, 17, 0, 70, 1])
    off = layout(counts, 1, 0)
    q, xs, w, ws = inputs(5, int(off[-1]), 7, 144, 272)
    out, err = run(q, xs, w, ws, "swiglu", counts, off, T, 2)
    assert err == 0
    check_experts(q, xs, w, ws, "swiglu", counts, off, out)


@pytest.mark.parametrize("T", [8, 100, 2000])
def test_rows_past_the_buffer_are_flagged(T):
    counts = np.array([30, 20, 10, 40])
    off = layout(counts, 1, 0)
    q, xs, w, ws = inputs(6, 100, 4, 64, 256)
    for cap in (75, 60, 45, 1):
        out, err = run(q, xs, w, ws, None, counts, off, T, 1, cap)
        assert err == moe.ERRBIT_EXPERT_CAP
        check_experts(q, xs, w, ws, None, counts, off, out)
    out, err = run(q, xs, w, ws, None, counts, off, T, 1)
    assert err == 0


@pytest.mark.parametrize("T", [10, 80, 300, 3000])
def test_counts_of_no_layout(T):
    """Counts and offsets that fit no buffer: nothing is written outside it."""
    q, xs, w, ws = inputs(7, 64, 3, 32, 64)
    big = 2 ** 31 - 1
    for counts, off in [([big, big, big], [0, big, big, big]), ([5, 5, 5], [-4, 0, 3, 1]),
                        ([-3, 4, 2], [0, 10, 20, 30]), ([4, 4, 4], [40, 30, 20, 10])]:
        run(q, xs, w, ws, None, counts, off, T, 1)


@pytest.mark.parametrize("T", [10, 300, 3000])
def test_counts_of_no_layout_of_many_experts(T):
    """More experts than a wave has lanes, all of them with the whole buffer."""
    E, big = 130, 2 ** 31 - 1
    q, xs, w, ws = inputs(8, 64, E, 32, 64)
    for counts, off in [([big] * E, [0] + [big] * E), ([64] * E, [-1] * (E + 1)),
                        ([1, -1] * (E // 2), list(range(E + 1)))]:
        run(q, xs, w, ws, None, counts, off, T, 1)


def test_numbers_of_rows_that_the_binding_is_given():
    """Without T all rows, whatever k; with T the first T * k."""
    q, xs, w, ws = inputs(12, 7, 1, 32, 64)
    whole, _ = run(q, xs, w, ws, None)
    out, _ = run(q, xs, w, ws, None, k=2)
    assert torch.equal(out, whole)
    out, _ = run(q, xs, w, ws, None, T=2, k=3)
    assert torch.equal(out[:6], whole[:6]) and bool((out[6:] == 0x5A5A).all())
    counts = np.array([3, 4])
    w2, ws2 = w.repeat(2, 1, 1), ws.repeat(2, 1)
    out, _ = run(q, xs, w2, ws2, None, counts, layout(counts, 1, 0), k=4)
    assert torch.equal(out, whole)


def test_a_slice_of_the_experts():
    counts = np.array([4, 9, 0, 33, 2, 80])
    off = layout(counts, 16, 0)
    q, xs, w, ws = inputs(8, int(off[-1]), 6, 48, 96)
    whole, _ = run(q, xs, w, ws, None, counts, off, int(counts.sum()), 1)
    for a, b in [(0, 2), (1, 4), (3, 6)]:
        out, err = run(q, xs, w[a:b], ws[a:b], None, counts[a:b], off[a:b + 1],
                       int(counts[a:b].sum()), 1)
        assert err == 0
        mine = torch.zeros(out.shape[0], dtype=torch.bool)
        for e in range(a, b):
            mine[off[e]:off[e] + counts[e]] = True
        mine = mine.cuda()
        assert torch.equal(out[mine], whole[mine]) and bool((out[~mine] == 0x5A5A).all())


@pytest.mark.parametrize("rows", [1, 20, 60, 100, 600])
def test_largest_sums(rows):
    """65,536 times -128 * -128 and 127 * -128: the ends of the sums."""
    K, N = 65536, 40
    q = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    w[0, 1::2] = 127
    q[::3] = 127
    xs, ws = torch.full((rows,), 2.0 ** -10, device="cuda"), torch.ones(1, N, device="cuda")
    out, _ = run(q, xs, w, ws, None)
    check(q, xs, w[0], ws[0], None, out.view(torch.bfloat16))


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_scales_that_are_not_finite_stay_in_their_row_and_column(rows):
    q, xs, w, ws = inputs(9, rows, 1, 64, 128)
    xs[1], xs[2], ws[0, 7] = float("nan"), float("inf"), float("nan")
    out, _ = run(q, xs, w, ws, None)
    out = out.view(torch.bfloat16)
    fine = torch.ones(rows, dtype=torch.bool)
    fine[1:3] = False
    cols = torch.ones(64, dtype=torch.bool)
    cols[7] = False
    fine, cols = fine.cuda(), cols.cuda()
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[:, 7]).all())
    assert not bool(torch.isfinite(out[2]).any())
    check(q[fine], xs[fine], w[0, cols], ws[0, cols], None, out[fine][:, cols])


def test_weights_far_into_their_tensor():
    """Experts whose weights lie behind the 2^31st byte, and rows that do."""
    E, N, K = 3, 16384, 65536
    w = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    g = gen(10)
    w[2, -40:] = codes(g, 40, K)
    ws = torch.ones(E, N, device="cuda")
    for rows in (3, 40, 100, 300):
        q, xs = codes(g, rows, K), torch.full((rows,), 2.0 ** -9, device="cuda")
        counts = np.array([0, 0, rows])
        out, err = run(q, xs, w, ws, None, counts, layout(counts, 1, 0), rows, 1)
        assert err == 0
        check(q, xs, w[2, -40:], ws[2, -40:], None, out[:, -40:].view(torch.bfloat16))
        assert bool((out[:, :-40] == 0).all())
    del w
    rows = 40000
    q = torch.zeros(rows, K, dtype=torch.int8, device="cuda")
    q[-3:] = codes(g, 3, K)
    xs = torch.full((rows,), 2.0 ** -9, device="cuda")
    w, ws = codes(g, 1, 33, K), torch.ones(1, 33, device="cuda")
    out, _ = run(q, xs, w, ws, None)
    check(q[-3:], xs[-3:], w[0], ws[0], None, out[-3:].view(torch.bfloat16))
    assert bool((out[:-3] == 0).all())


def test_gates_far_from_their_other_factors():
    """Gates and other factors more than 2^31 bytes apart."""
    N, K = 1 << 17, 32768
    half = N // 2
    g = gen(11)
    w = torch.zeros(1, N, K, dtype=torch.int8, device="cuda")
    w[0, half - 50:half], w[0, N - 50:] = codes(g, 50, K), codes(g, 50, K)
    ws = torch.full((1, N), 2.0 ** -8, device="cuda")
    pick = torch.cat([torch.arange(half - 50, half), torch.arange(N - 50, N)]).cuda()
    for rows in (1, 20, 60, 200, 1000):
        say(f"far gates rows={rows}")
        q, xs = codes(g, rows, K), torch.full((rows,), 2.0 ** -9, device="cuda")
        out, _ = run(q, xs, w, ws, "swiglu")
        check(q, xs, w[0, pick], ws[0, pick], "swiglu", out[:, -50:].view(torch.bfloat16))
        assert bool((out[:, :-50] == 0).all())


def test_two_streams_at_once_and_a_graph():
    """Calls on two streams at once, and a captured one replayed with new rows,
    give what each gives alone."""
    N, K = 512, 1024
    sets = [inputs(20 + i, r, 1, N, K) for i, r in enumerate((9, 700))]
    alone = [run(*s, "swiglu")[0] for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros_like(a) for a in alone] for _ in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                moe.int8_product(*sets[i], o[i], act="swiglu")
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(alone, o))
    q, xs, w, ws = (t.clone() for t in sets[1])
    out, mid = torch.zeros_like(alone[1]), torch.empty(700, N // 2, device="cuda",
                                                       dtype=torch.bfloat16)
    q2, s2 = torch.empty(700, N // 2, dtype=torch.int8, device="cuda"), torch.empty(700,
                                                                                    device="cuda")
    w2, ws2 = codes(gen(3), 1, N // 2, N // 2), torch.ones(1, N // 2, device="cuda") / 4096

    def step(to):
        moe.int8_product(q, xs, w, ws, mid, act="swiglu")
        moe.quantise_rows(mid, q2, s2)
        moe.int8_product(q2, s2, w2, ws2, to)

    step(out)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(out)
    for n in range(4):
        q.copy_(codes(gen(40 + n), 700, K))
        out.zero_()
        graph.replay()
        if n % 2:
            torch.cuda.synchronize()
        want = torch.zeros_like(out)
        step(want)
        torch.cuda.synchronize()
        assert torch.equal(out, want), n
