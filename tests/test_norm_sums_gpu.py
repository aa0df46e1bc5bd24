"""The norm's weight gradient where a thread adds up many rows, on the GPU against
64 bits.

A thread adds up at most 16 rows in one float32 value, then adds this to two of
them: what the addition to the first rounds off goes to the second, whose own roundings
come to less than 2^-24 of the sum of the terms' magnitudes as long as a thread has
fewer than 65,536 rows (16 * 4,096: 4,096 additions of at most 4,096 * 2^-24 of it, each
rounded by 2^-24). So the error does not grow with the number of rows. In ULP = 2^-24 of
the sum of magnitudes: sum * inv_rms 1, the 16 additions 16, the second value's roundings
1, the two made one 1, an addition in float32 for each further row that a workgroup takes
at a time; of the result: 1, rounded from 64 bits."""
import pytest
import torch

import combine_topk_ids_02_amd as moe

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24
F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


def weight_gradient(d, h, inv):
    T, H = d.shape
    got = torch.empty(H, device="cuda")
    ws = torch.empty(moe.norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.norm_backward(d, h, inv, torch.ones(H, device="cuda"), d_weight=got, workspace=ws)
    torch.cuda.synchronize()
    return got


def check(d, h, inv, at_once):
    got = weight_gradient(d, h, inv).to(F64)
    want, most = torch.zeros_like(got), torch.zeros_like(got)
    step = max(1, (1 << 26) // d.shape[1])
    for a in range(0, d.shape[0], step):
        b = slice(a, a + step)
        terms = d[b].to(F64) * (h[b].to(F64) * inv[b].to(F64)[:, None])
        want += terms.sum(dim=0)
        most += terms.abs().sum(dim=0)
    bound = ULP * ((19 + at_once - 1) * most + want.abs())
    off = (got - want).abs()
    print("most of its bound", float((off / bound).max()), flush=True)
    assert bool((off <= bound).all())


# rows, their width, and how many of them a workgroup takes at a time
CASES = [(1 << 23, 8, 16, BF), (1 << 23, 8, 16, F32), (1 << 20, 520, 8, BF),
         ((1 << 16) - 5, 5120, 1, BF), ((1 << 16) + 3, 5120, 1, F32), (1 << 15, 16384, 1, BF),
         (1 << 15, 32768, 1, F32)]


@pytest.mark.parametrize("T, H, at_once, stream", CASES)
@pytest.mark.parametrize("kind", ["equal", "positive", "any"])
def test_weight_gradient_of_many_rows(T, H, at_once, stream, kind):
    print(f"[rows] {T} x {H} {stream} {kind}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    if kind == "equal":
        d = torch.full((T, H), 1.0078125, dtype=BF, device="cuda")
        h = torch.ones(T, H, dtype=stream, device="cuda")
        inv = torch.full((T,), 0.7, device="cuda")
    else:
        d = torch.randn(T, H, dtype=BF, device="cuda", generator=g)
        h = torch.randn(T, H, dtype=stream, device="cuda", generator=g)
        inv = 0.5 + torch.rand(T, device="cuda", generator=g)
        if kind == "positive":
            d, h = d.abs_(), h.abs_()
    check(d, h, inv, at_once)


@pytest.mark.parametrize("stream", [BF, F32])
def test_weight_gradient_that_is_not_finite(stream):
    """An infinity or a NaN of d_out, and a sum past float32, stay in their columns."""
    T, H = 30000, 16
    d = torch.ones(T, H, dtype=BF, device="cuda")
    h = torch.ones(T, H, dtype=stream, device="cuda")
    inv = torch.ones(T, device="cuda")
    for row in (0, 9000, T - 1):
        d[row, 1], d[row, 2], d[row, 3] = float("inf"), float("-inf"), float("nan")
    d[:, 4], d[:, 5] = 3e38, -3e38
    got = weight_gradient(d, h, inv)
    assert float(got[1]) == float("inf") and float(got[2]) == float("-inf")
    assert bool(torch.isnan(got[3]))
    assert float(got[4]) == float("inf") and float(got[5]) == float("-inf")
    assert bool((got[[0] + list(range(6, H))] == T).all())


@pytest.mark.parametrize("T, H, stream", [(9001, 5120, F32), (9001, 10240, BF), (140000, 64, BF)])
def test_many_rows_in_a_graph(T, H, stream):
    """Replayed on a workspace of NaNs, with eager calls between: the same to the bit."""
    print(f"[graph] {T} x {H} {stream}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    d = torch.randn(T, H, dtype=BF, device="cuda", generator=g)
    h = torch.randn(T, H, dtype=stream, device="cuda", generator=g)
    inv, ones = 0.5 + torch.rand(T, device="cuda", generator=g), torch.ones(H, device="cuda")
    got = torch.empty(H, device="cuda")
    room = torch.empty(moe.norm_workspace_bytes(T, H) // 4, device="cuda")

    def step():
        moe.norm_backward(d, h, inv, ones, d_weight=got, workspace=room)

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for n in range(4):
        d.mul_(-1)
        want = weight_gradient(d, h, inv)
        got.zero_()
        room.fill_(float("nan"))
        graph.replay()
        if n % 2:
            torch.cuda.synchronize()
        assert torch.equal(got, want), n
