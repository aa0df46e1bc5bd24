"""A layer in 8-bit integers, as its calls are used together: the norm with the
residual's addition, the router, the dispatch, the experts' rows to int8, their two
products with the quantiser between them, the combine, and the shared expert on the
norm's own int8 rows; and a training step of the norm. Every step is checked on what
the step before it left: a code against half a step of its row, a product without an
activation to the bit, the others by half a step of bf16 (2^-8) and the roundings of
float32 (2^-24 each) that the formula takes."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe

pytestmark = pytest.mark.gpu
F64, BF = torch.float64, torch.bfloat16
ULP, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


class Layer:
    def __init__(self, T, H, I, E, R, k, seed, align=1, block=0, stream=torch.float32):
        g = self.g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.T, self.H, self.I, self.E, self.R, self.k = T, H, I, E, R, k
        self.align, self.block = align, block
        dev = torch.device("cuda:0")
        b = self.b = moe.Buffers(moe.Shape(T, H, E, R, k, align, block), dev)
        cap = b.expert_buf.shape[0]

        def z(dtype, *shape):
            return torch.zeros(shape, dtype=dtype, device=dev)

        def codes(*shape):
            return torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8)

        def scales(*shape):
            return (0.5 + torch.rand(*shape, generator=g, device=dev)) / (64 * shape[-1] ** 0.5)

        self.w1, self.s1 = codes(E, 2 * I, H), scales(E, 2 * I)
        self.w2, self.s2 = codes(E, H, I), scales(E, H)
        self.v1, self.t1 = codes(1, 2 * I, H), scales(1, 2 * I)
        self.v2, self.t2 = codes(1, H, I), scales(1, H)
        self.gain = 1 + 0.1 * torch.randn(H, generator=g, device=dev)
        self.x, self.res, self.sum = z(BF, T, H), z(stream, T, H), z(stream, T, H)
        self.normed, self.inv = z(BF, T, H), z(torch.float32, T)
        self.xq, self.xs = z(torch.int8, T, H), z(torch.float32, T)
        self.logits, self.ids = z(torch.float32, T, E), z(torch.int32, T, k)
        self.weights = z(torch.float32, T, k)
        self.eq, self.es = z(torch.int8, cap, H), z(torch.float32, cap)
        self.mid, self.mq, self.ms = z(BF, cap, I), z(torch.int8, cap, I), z(torch.float32, cap)
        self.expert_out = z(BF, cap, H)
        self.smid, self.sq, self.ss = z(BF, T, I), z(torch.int8, T, I), z(torch.float32, T)
        self.shared = z(BF, T, H)
        self.router = moe.Router("sigmoid", True, 1.0)

    def fill(self):
        for t in (self.x, self.res, self.logits):
            t.copy_(torch.randn(t.shape, device="cuda", generator=self.g))

    def forward(self):
        b = self.b
        moe.norm(self.x, self.gain, residual=self.res, sum=self.sum, out=self.normed, fmt="int8",
                 q=self.xq, q_scale=self.xs, inv_rms=self.inv)
        moe.route(self.logits, self.k, self.router, self.ids, self.weights, err=b.err)
        moe.dispatch_all(self.normed, self.ids, self.E, self.R, b.layout_dict(), b.rank_buf,
                         b.rank_src_token, b.expert_buf, b.expert_src_pair, align=self.align,
                         block=self.block, workspace=b.workspace, err=b.err)
        moe.quantise_rows(b.expert_buf, self.eq, self.es, pair_row=b.pair_row, err=b.err)
        runs = dict(expert_counts=b.expert_counts, expert_offsets=b.expert_offsets, T=self.T,
                    k=self.k, err=b.err)
        moe.int8_product(self.eq, self.es, self.w1, self.s1, self.mid, act="swiglu", **runs)
        moe.quantise_rows(self.mid, self.mq, self.ms, pair_row=b.pair_row, err=b.err)
        moe.int8_product(self.mq, self.ms, self.w2, self.s2, self.expert_out, **runs)
        moe.combine(self.expert_out, b.pair_row, self.weights, self.E, self.R, b.out, err=b.err)
        moe.int8_product(self.xq, self.xs, self.v1, self.t1, self.smid, act="swiglu")
        moe.quantise_rows(self.smid, self.sq, self.ss)
        moe.int8_product(self.sq, self.ss, self.v2, self.t2, self.shared)

    def outputs(self):
        return [self.sum, self.normed, self.xq, self.xs, self.inv, self.b.out, self.shared,
                self.expert_out, self.mid]


def check_codes(v, q, s):
    """q * s against v: half a step, and the roundings of the scale, the factor and
    the products."""
    v = v.to(F64)
    top = v.abs().amax(dim=1, keepdim=True)
    off = (q.to(F64) * s.to(F64)[:, None] - v).abs()
    assert bool((off <= top / 127 * (0.5 + 127 * 6 * ULP)).all())


def check_product(q, s, w, ws, act, got):
    y = q.to(F64) @ w.to(F64).t().contiguous()
    if not act:
        assert torch.equal(got, (y.to(torch.float32) * s[:, None] * ws).to(BF))
        return
    y = y * s.to(F64)[:, None] * ws.to(F64)
    n = y.shape[1] // 2
    gate, up = y[:, :n], y[:, n:]
    want = gate * torch.sigmoid(gate) * up
    bound = ULP * (3.3 * (gate * up).abs() + 13 * want.abs()) + HALF * want.abs() + 1e-38
    assert bool(((got.to(F64) - want).abs() <= bound).all())


def check(layer):
    a, b = layer, layer.b
    assert int(b.err.item()) == 0
    s = (a.x.float() + a.res.float()).to(a.res.dtype)
    assert torch.equal(a.sum, s)
    y = s.to(F64) / torch.sqrt(s.to(F64).square().mean(dim=1, keepdim=True) + 1e-6) * a.gain
    assert bool(((a.normed.to(F64) - y).abs() <= (HALF + 38 * ULP) * y.abs() + 1e-40).all())
    top = y.abs().amax(dim=1, keepdim=True)
    off = (a.xq.to(F64) * a.xs.to(F64)[:, None] - y).abs()
    assert bool((off <= top / 127 * (0.5 + 127 * 100 * ULP)).all())
    counts, offsets = b.expert_counts.tolist(), b.expert_offsets.tolist()
    for e in range(a.E):
        r = slice(offsets[e], offsets[e] + counts[e])
        if counts[e] == 0:
            continue
        check_codes(b.expert_buf[r], a.eq[r], a.es[r])
        check_product(a.eq[r], a.es[r], a.w1[e], a.s1[e], True, a.mid[r])
        check_codes(a.mid[r], a.mq[r], a.ms[r])
        check_product(a.mq[r], a.ms[r], a.w2[e], a.s2[e], False, a.expert_out[r])
    rows = a.expert_out[b.pair_row.long()].to(F64)
    terms = rows * a.weights.to(F64)[:, :, None]
    want = terms.sum(dim=1)
    bound = HALF * want.abs() + (a.k + 1) * ULP * terms.abs().sum(dim=1) * (1 + HALF) + 1e-40
    assert bool(((b.out.to(F64) - want).abs() <= bound).all())
    check_product(a.xq, a.xs, a.v1[0], a.t1[0], True, a.smid)
    check_codes(a.smid, a.sq, a.ss)
    check_product(a.sq, a.ss, a.v2[0], a.t2[0], False, a.shared)


CASES = [(1, 512, 256, 16, 4, 4, 1, 0), (64, 1024, 96, 64, 8, 6, 1, 0),
         (37, 512, 160, 32, 4, 8, 16, 0), (130, 256, 64, 16, 2, 3, 1, 130),
         (700, 256, 144, 8, 2, 5, 128, 0)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("stream", [BF, torch.float32])
def test_layer(case, stream):
    T, H, I, E, R, k, align, block = CASES[case]
    print(f"[layer] {CASES[case]} {stream}", flush=True)
    layer = Layer(T, H, I, E, R, k, 50 + case, align, block, stream)
    layer.fill()
    layer.forward()
    torch.cuda.synchronize()
    check(layer)


def test_layer_in_a_graph():
    """Captured once, replayed with new inputs; every replay equals the eager step,
    with the program's own work between them."""
    layer = Layer(64, 512, 96, 64, 8, 6, 60, align=16)
    layer.fill()
    layer.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward()
    for n in range(4):
        layer.fill()
        layer.forward()
        torch.cuda.synchronize()
        check(layer)
        want = [t.clone() for t in layer.outputs()]
        for t in layer.outputs()[:-2]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, exp in zip(layer.outputs(), want):
            assert torch.equal(got, exp), n


def test_layers_on_two_streams():
    """Two layers at once give what each gives alone."""
    layers = [Layer(96, 512, 128, 32, 4, 4, 70 + i, block=96) for i in range(2)]
    for layer in layers:
        layer.fill()
        layer.forward()
    torch.cuda.synchronize()
    want = [[t.clone() for t in layer.outputs()] for layer in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for layer, st in zip(layers, streams):
            with torch.cuda.stream(st):
                layer.forward()
    torch.cuda.synchronize()
    for layer, exp in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(layer.outputs(), exp))


def test_training_step_of_two_norms():
    """h1 = h0 + f0, y1 = norm(h1), h2 = h1 + y1, y2 = norm(h2) and the loss
    sum(c2 * y2): the gradients of h0 and both weights by two calls, the second's
    stream gradient passing on to the first, against central differences in 64 bits.
    The stream is float32 and y1 is passed on in bf16, so the second norm's gradient
    of its x (bf16) is off by 2^-8 of itself; the differences take the loss as the
    function of the float32 stream that the kernels see."""
    g = torch.Generator()
    g.manual_seed(80)
    T, H = 3, 64
    h0, f0 = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g).to(BF)
    w1, w2 = (1 + 0.1 * torch.randn(H, generator=g) for _ in range(2))
    c2 = torch.randn(T, H, generator=g).to(BF)
    dev = "cuda"

    def new(dtype, *s):
        return torch.zeros(s, dtype=dtype, device=dev)

    h1, y1, i1 = new(torch.float32, T, H), new(BF, T, H), new(torch.float32, T)
    h2, y2, i2 = new(torch.float32, T, H), new(BF, T, H), new(torch.float32, T)
    moe.norm(f0.cuda(), w1.cuda(), residual=h0.cuda(), sum=h1, out=y1, inv_rms=i1)
    moe.norm(y1, w2.cuda(), residual=h1, sum=h2, out=y2, inv_rms=i2)
    ws = torch.empty(moe.norm_workspace_bytes(T, H), dtype=torch.uint8, device=dev)
    dy1, dh1, dw2 = new(BF, T, H), new(torch.float32, T, H), new(torch.float32, H)
    moe.norm_backward(c2.cuda(), h2, i2, w2.cuda(), d_x=dy1, d_residual=dh1, d_weight=dw2,
                      workspace=ws)
    dh0, df0, dw1 = new(torch.float32, T, H), new(BF, T, H), new(torch.float32, H)
    moe.norm_backward(dy1, h1, i1, w1.cuda(), d_sum=dh1, d_x=df0, d_residual=dh0, d_weight=dw1,
                      workspace=ws)
    torch.cuda.synchronize()

    def unit(h):
        return h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + 1e-6)

    def loss(a, u, v):
        b = a + f0.to(F64)
        c = b + unit(b) * u
        return (c2.to(F64) * unit(c) * v).sum().item()

    a, u, v = h0.to(F64), w1.to(F64), w2.to(F64)
    step = 1e-5
    # the second call's bf16 gradient is off by half a step of its values, and y1 by
    # half a step of its own; both pass on to the first with the size of that norm's
    # Jacobian, |w| / rms (1 + 1), and of the second's
    size = float((w1.abs().max() * i1.abs().max() * 2).item())
    most = float(dy1.float().abs().max())
    slack = HALF * most * size * 2 + 2 * HALF * float(y1.float().abs().max()) * most * size
    for r, c in [(0, 0), (1, 17), (2, 63), (2, 5)]:
        e = torch.zeros(T, H, dtype=F64)
        e[r, c] = step
        slope = (loss(a + e, u, v) - loss(a - e, u, v)) / (2 * step)
        assert abs(slope - float(dh0[r, c])) <= slack
        assert abs(float(df0[r, c]) - float(dh0[r, c])) <= HALF * abs(float(dh0[r, c]))
        f = torch.zeros(H, dtype=F64)
        f[c] = step
        slope = (loss(a, u + f, v) - loss(a, u - f, v)) / (2 * step)
        terms = float(dy1.float()[:, c].abs().sum() * 8)  # |unit| is at most sqrt(64)
        assert abs(slope - float(dw1[c])) <= 2 * HALF * terms + slack
        slope = (loss(a, u, v + f) - loss(a, u, v - f)) / (2 * step)
        terms = float(c2.float()[:, c].abs().sum() * 8)
        assert abs(slope - float(dw2[c])) <= 2 * HALF * terms


@pytest.mark.parametrize("fast", [True, False])
def test_binding_refuses_wrong_tensors(fast, monkeypatch):
    """With the binding's C++ part and without it."""
    if not fast:
        monkeypatch.setattr(moe, "_fast", None)
        monkeypatch.setattr(moe, "_address", None)
    dev = "cuda"
    x, w = torch.zeros(4, 64, dtype=BF, device=dev), torch.zeros(64, device=dev)
    f = torch.zeros(4, 64, device=dev)
    q, s = torch.zeros(4, 64, dtype=torch.int8, device=dev), torch.zeros(4, device=dev)
    inv = torch.zeros(4, device=dev)
    wq, wsc = torch.zeros(1, 32, 64, dtype=torch.int8, device=dev), torch.zeros(1, 32, device=dev)
    out = torch.zeros(4, 32, dtype=BF, device=dev)
    ids = torch.zeros(4, 1, dtype=torch.int32, device=dev)
    bad = [
        lambda: moe.norm(f, w, out=x), lambda: moe.norm(x, w.half(), out=x),
        lambda: moe.norm(x, w[:32], out=x), lambda: moe.norm(x, w, out=x[:, :32]),
        lambda: moe.norm(x, w, out=f), lambda: moe.norm(x, w), lambda: moe.norm(x, w, residual=x),
        lambda: moe.norm(x, w, residual=x, sum=f, out=x),
        lambda: moe.norm(x, w, residual=x.half(), sum=x.half(), out=x),
        lambda: moe.norm(x, w, out=x, fmt="fp8"), lambda: moe.norm(x, w, out=x, fmt="int8"),
        lambda: moe.norm(x, w, fmt="int8", q=q.view(torch.uint8), q_scale=s),
        lambda: moe.norm(x, w, fmt="mxfp8", q=q, q_scale=s), lambda: moe.norm(x, w, out=x, eps=0.0),
        lambda: moe.norm(x, w, out=x, q=q, q_scale=s),
        lambda: moe.norm(x, w, out=x, inv_rms=inv[:3]),
        lambda: moe.norm(x[:, ::2], w[:32], out=x[:, :32].contiguous()),
        lambda: moe.norm_backward(x, f, inv, w), lambda: moe.norm_backward(f, f, inv, w, d_x=x),
        lambda: moe.norm_backward(x, f, inv, w, d_x=f),
        lambda: moe.norm_backward(x, f, inv, w, d_residual=x),
        lambda: moe.norm_backward(x, f, inv, w, d_x=x, d_sum=x),
        lambda: moe.norm_backward(x, f, inv, w, d_weight=w),
        lambda: moe.norm_backward(x, f, inv, w, d_weight=w, workspace=inv),
        lambda: moe.quantise_rows(f, q, s), lambda: moe.quantise_rows(x, q, s[:3]),
        lambda: moe.quantise_rows(x, q.view(torch.uint8), s),
        lambda: moe.quantise_rows(x, q, s, pair_row=ids.long()),
        lambda: moe.quantise_rows(x, q, s, pair_row=ids[:, 0]),
        lambda: moe.int8_product(x, s, wq, wsc, out), lambda: moe.int8_product(q, s, wq, wsc, x),
        lambda: moe.int8_product(q, s, wq, wsc, out, act="swiglu"),
        lambda: moe.int8_product(q, s, wq, wsc[0], out),
        lambda: moe.int8_product(q, s, wq, wsc, out, T=5),
        lambda: moe.int8_product(q, s, wq, wsc, out, expert_counts=ids[0]),
        lambda: moe.int8_product(q, s, wq.expand(2, 32, 64).contiguous(), wsc.repeat(2, 1), out),
        lambda: moe.int8_product(q, s, wq.float(), wsc, out),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(moe.MoeError):
            call()
            print("accepted:", n)
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x.copy_(torch.randn(4, 64, device=dev, generator=g))
    w += 1
    moe.norm(x, w, fmt="int8", q=q, q_scale=s, inv_rms=inv)
    wsc += 1
    wq += 1
    moe.int8_product(q, s, wq, wsc, out)
    want = (q.float().sum(dim=1) * s).to(BF)
    assert torch.equal(out, want[:, None].expand(4, 32))
