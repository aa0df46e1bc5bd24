"""An MoE layer from router logits to its output, as a decode step runs it
(route, moe_dispatch, the two expert products, combine), and a router's
training step (route, balance loss, both gradients): against the 64-bit
formulas, captured into a HIP graph and replayed with new inputs, and on two
streams at once."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe
import router_ref as ref
from router_ref import ULP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


class Layer:
    """Buffers and weights of one layer; forward() is a decode step."""

    def __init__(self, T, H, I, E, R, k, fmt, seed, align=1, block=0):
        rng = np.random.default_rng(seed)
        blk = 32 if fmt == "mxfp4" else 16
        self.T, self.H, self.I, self.E, self.R, self.k, self.fmt = T, H, I, E, R, k, fmt
        self.align, self.block = align, block
        dev = torch.device("cuda:0")
        self.b = moe.Buffers(moe.Shape(T, H, E, R, k, align, block), dev)
        lo, hi = (118, 122) if fmt == "mxfp4" else (16, 28)

        def scales(n, w):
            return rng.integers(lo, hi, size=(E, n, w // blk)).astype(np.uint8)

        self.q1 = rng.integers(0, 256, size=(E, 2 * I, H // 2)).astype(np.uint8)
        self.s1 = scales(2 * I, H)
        self.q2 = rng.integers(0, 256, size=(E, H, I // 2)).astype(np.uint8)
        self.s2 = scales(H, I)
        self.w = [torch.from_numpy(a).cuda() for a in (self.q1, self.s1, self.q2, self.s2)]
        cap = self.b.expert_buf.shape[0]
        self.mid = torch.zeros(cap, I, dtype=torch.bfloat16, device=dev)
        self.expert_out = torch.zeros(cap, H, dtype=torch.bfloat16, device=dev)
        self.router = moe.Router("sigmoid", True, 2.5, 4, 2)
        self.bias = torch.from_numpy(rng.normal(size=E).astype(np.float32) * 0.1).cuda()
        self.ids = torch.zeros(T, k, dtype=torch.int32, device=dev)
        self.weights = torch.zeros(T, k, device=dev)
        self.logits = torch.zeros(T, E, device=dev)
        self.hidden = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.logits.copy_(torch.randn(self.T, self.E, device="cuda", generator=g))
        self.hidden.copy_(torch.randn(self.T, self.H, device="cuda", generator=g))

    def forward(self):
        b = self.b
        moe.route(self.logits, self.k, self.router, self.ids, self.weights, bias=self.bias,
                  err=b.err)
        moe.dispatch_all(self.hidden, self.ids, self.E, self.R, b.layout_dict(), b.rank_buf,
                         b.rank_src_token, b.expert_buf, b.expert_src_pair, align=self.align,
                         block=self.block, workspace=b.workspace, err=b.err)
        moe.expert_product(self.fmt, b.expert_buf, b.expert_counts, b.expert_offsets, self.T,
                           self.k, self.w[0], self.w[1], self.mid, act="swiglu", err=b.err)
        moe.expert_product(self.fmt, self.mid, b.expert_counts, b.expert_offsets, self.T, self.k,
                           self.w[2], self.w[3], self.expert_out, err=b.err)
        moe.combine(self.expert_out, b.pair_row, self.weights, self.E, self.R, b.out, err=b.err)
        return b.out

    def expected(self):
        """(output in 64 bits, tolerance): mid, expert_out and the output are
        each rounded to bf16 once (half a step, 2^-8), and each sum over n
        values is off by at most n / 4 + 8 roundings of its absolute terms."""
        z = self.logits.double().cpu().numpy()
        x = self.hidden.double().cpu().numpy()
        ids, _ = ref.choose(z, self.k, "sigmoid", self.bias.cpu().numpy(), 4, 2)
        w = ref.weights(z, ids, "sigmoid", True, 2.5)
        out, tol = np.zeros((self.T, self.H)), np.zeros((self.T, self.H))
        half = 2.0 ** -8
        for e in range(self.E):
            at = np.argwhere(ids == e)
            if at.size == 0:
                continue
            t, j = at[:, 0], at[:, 1]
            w1 = ref.weight_values(self.fmt, self.q1[e], self.s1[e])
            w2 = ref.weight_values(self.fmt, self.q2[e], self.s2[e])
            y, ty = x[t] @ w1.T, (abs(x[t]) @ abs(w1.T)) * (self.H / 4 + 8) * ULP
            g, u = y[:, :self.I], y[:, self.I:]
            silu = g * ref.sigmoid(g)
            mid = silu * u
            tm = 1.1 * ty[:, :self.I] * (abs(u) + ty[:, self.I:]) + abs(silu) * ty[:, self.I:]
            tm = tm + abs(mid) * (half + 16 * ULP * (1 + abs(g)))
            y2 = mid @ w2.T
            t2 = tm @ abs(w2.T) + (abs(mid) @ abs(w2.T)) * (self.I / 4 + 8) * ULP
            t2 = t2 * (1 + half) + half * abs(y2)
            out[t] += w[t, j][:, None] * y2
            tol[t] += w[t, j][:, None] * (t2 * (1 + half) + 64 * ULP * abs(y2))
        return ids, out, tol + half * (abs(out) + tol)


CASES = [(1, 512, 256, 16, 4, 4, "mxfp4", 1, 0), (64, 512, 96, 64, 8, 6, "nvfp4", 1, 0),
         (37, 1024, 160, 32, 4, 8, "mxfp4", 16, 0), (130, 256, 64, 16, 2, 3, "nvfp4", 1, 130),
         (300, 256, 64, 16, 2, 5, "mxfp4", 1, 0)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode_layer(case):
    T, H, I, E, R, k, fmt, align, block = CASES[case]
    print(f"[layer] {CASES[case]}", flush=True)
    layer = Layer(T, H, I, E, R, k, fmt, 30 + case, align, block)
    layer.fill(1)
    out = layer.forward()
    torch.cuda.synchronize()
    ids, want, tol = layer.expected()
    assert int(layer.b.err.item()) == 0
    assert np.array_equal(layer.ids.cpu().numpy(), ids)
    assert (abs(out.double().cpu().numpy() - want) <= tol).all()


def test_decode_layer_in_a_graph():
    """Captured once, replayed with new logits and hidden states; every replay
    equals the eager step, with the program's own work between them."""
    layer = Layer(64, 512, 96, 64, 8, 6, "mxfp4", 40)
    layer.fill(1)
    layer.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward()
    for seed in range(2, 7):
        layer.fill(seed)
        layer.forward()
        torch.cuda.synchronize()
        want = [layer.b.out.clone(), layer.ids.clone(), layer.weights.clone()]
        layer.b.out.zero_()
        layer.ids.fill_(-3)
        layer.weights.zero_()
        layer.expert_out.zero_()
        layer.mid.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, exp in zip((layer.b.out, layer.ids, layer.weights), want):
            assert torch.equal(got, exp), seed
    assert int(layer.b.err.item()) == 0


def test_decode_layers_on_two_streams():
    """Two layers at once on two streams give what each gives alone."""
    layers = [Layer(64, 512, 96, 64, 8, 6, "mxfp4", 41), Layer(48, 512, 128, 32, 4, 4, "nvfp4", 42)]
    want = []
    for i, layer in enumerate(layers):
        layer.fill(i)
        want.append(layer.forward().clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                layer.b.out.zero_()
                for _ in range(3):
                    layer.forward()
        torch.cuda.synchronize()
        for layer, exp in zip(layers, want):
            assert torch.equal(layer.b.out, exp)


class Training:
    """A router's training step: choice and weights, the balance losses and the
    gradient of <weights, d_weights> + <loss, d_loss>."""

    def __init__(self, T, E, k, scoring, S, dtype, seed):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.S, self.scoring = T, E, k, S, scoring
        self.router = moe.Router(scoring)
        cuda = dict(device="cuda")
        self.logits = torch.zeros(T, E, dtype=dtype, **cuda)
        self.ids = torch.zeros(T, k, dtype=torch.int32, **cuda)
        self.weights = torch.zeros(T, k, **cuda)
        self.out = [torch.zeros(S, **cuda), torch.zeros(S, E, dtype=torch.int32, **cuda),
                    torch.zeros(S, dtype=torch.int32, **cuda), torch.zeros(S, E, **cuda)]
        self.ws = torch.empty(moe.balance_workspace_bytes(T, E, k, S), dtype=torch.uint8, **cuda)
        cut = np.sort(rng.integers(0, T + 1, size=S - 1))
        self.off = np.concatenate([[0], cut, [T - T // 10]]).astype(np.int32)
        self.off = np.minimum(self.off, T - T // 10)
        self.off_d = torch.from_numpy(self.off).cuda()
        self.mask = torch.arange(T, device="cuda") < T - T // 20
        self.dw = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda()
        self.dl = torch.from_numpy(rng.normal(size=S).astype(np.float32)).cuda()
        self.dz = torch.zeros(T, E, dtype=dtype, **cuda)
        self.err = torch.zeros(1, dtype=torch.int32, **cuda)

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.logits.copy_(torch.randn(self.T, self.E, device="cuda", generator=g))

    def step(self):
        moe.route(self.logits, self.k, self.router, self.ids, self.weights,
                  token_mask=self.mask, err=self.err)
        moe.balance_loss(self.logits, self.ids, self.router, *self.out, seq_offsets=self.off_d,
                         workspace=self.ws, err=self.err)
        moe.route_backward(self.logits, self.ids, self.router, self.dz, d_weights=self.dw,
                           balance=(self.dl, self.out[1], self.out[2], self.off_d), err=self.err)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_training_step(scoring):
    T, E, k, S = 700, 96, 6, 5
    tr = Training(T, E, k, scoring, S, torch.float32, 50)
    tr.fill(3)
    tr.step()
    torch.cuda.synchronize()
    z = tr.logits.double().cpu().numpy()
    mask = tr.mask.cpu().numpy()
    ids, _ = ref.choose(z, k, scoring, mask=mask)
    assert int(tr.err.item()) == 0
    assert np.array_equal(tr.ids.cpu().numpy(), ids)
    loss, counts, tokens, mean = ref.balance(z, ids, scoring, tr.off)
    got = [o.cpu().numpy() for o in tr.out]
    assert np.array_equal(got[1], counts) and np.array_equal(got[2], tokens)
    # logits of N(0, 1): spreads below 12; counted as in test_router_gpu.py
    assert (abs(got[0] - loss) <= 90 * ULP * loss).all()
    assert (abs(got[3] - mean) <= 90 * ULP * mean).all()
    want, size = ref.gradient(z, ids, scoring, True, 1.0, tr.dw.cpu().numpy(), tr.dl.cpu().numpy(),
                              tr.off)
    assert (abs(tr.dz.double().cpu().numpy() - want) <= 90 * ULP * size + 1e-37).all()


def test_training_step_in_a_graph():
    """Replays with new logits equal eager steps, bit for bit, while the eager
    program keeps working on the same tensors in between."""
    tr = Training(3000, 256, 8, "sigmoid", 7, torch.bfloat16, 51)
    tr.fill(1)
    tr.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.step()
    for seed in range(2, 6):
        tr.fill(seed)
        tr.step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (tr.ids, tr.weights, *tr.out, tr.dz)]
        tr.dz.fill_(9)
        tr.ids.fill_(-5)
        for o in tr.out:
            o.fill_(3)
        tr.ws.fill_(0x33)
        graph.replay()
        torch.cuda.synchronize()
        for got, exp in zip((tr.ids, tr.weights, *tr.out, tr.dz), want):
            assert torch.equal(got, exp), seed
    assert int(tr.err.item()) == 0


def test_binding_refuses_wrong_tensors():
    z = torch.zeros(8, 16, device="cuda")
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(8, 2, device="cuda")
    r = moe.Router()
    ok = dict(logits=z, k=2, router=r, topk_ids=ids, topk_weights=w)
    moe.route(**ok)
    for bad in (dict(logits=z[:, :8]), dict(topk_ids=ids.long()), dict(topk_ids=ids.cpu()),
                dict(topk_weights=w[:7]), dict(bias=z[0]), dict(token_mask=w[:, 0]),
                dict(err=w), dict(err=ids[:0, 0]), dict(k=3), dict(k=0),
                dict(bias=z[:, 0], router=moe.Router("sigmoid"))):
        with pytest.raises(moe.MoeError):
            moe.route(**{**ok, **bad})
    with pytest.raises(moe.MoeError):
        moe.route_backward(z, ids, r, z.to(torch.bfloat16), d_weights=w)
    with pytest.raises(moe.MoeError):
        moe.route_backward(z, ids, r, torch.empty_like(z))
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    cnt = torch.zeros(1, 16, dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoeError):  # the workspace is too small
        moe.balance_loss(z, ids, r, w[0, :1], cnt, cnt[0, :1], z[:1], workspace=ws)
    rows = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 4, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 4, 2, dtype=torch.uint8, device="cuda")
    counts = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    out = torch.zeros(8, 4, dtype=torch.bfloat16, device="cuda")
    moe.expert_product("mxfp4", rows, counts, off, 8, 1, q, s, out)
    for args in (("nvfp4", rows, counts, off, 8, 1, q, s, out),
                 ("mxfp4", rows, counts, off[:2], 8, 1, q, s, out),
                 ("mxfp4", rows, counts, off, 8, 1, q, s, out[:, :2]),
                 ("mxfp4", rows, counts, off, 8, 1, q.int(), s, out),
                 ("mxfp4", rows[:, ::2], counts, off, 8, 1, q, s, out),
                 ("mxfp4", rows, counts, off, -1, 1, q, s, out),
                 ("mxfp4", rows.float(), counts, off, 8, 1, q, s, out)):
        with pytest.raises(moe.MoeError):
            moe.expert_product(*args)
