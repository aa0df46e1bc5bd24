"""The norm, its gradient and the rows' quantiser on the GPU against their
formulas in 64 bits.

Tolerances, in half steps of float32 (ULP = 2^-24): a row's sum runs through at
most 4 pieces of 8 values a lane, 6 steps over the wave and 16 waves, so a sum of
terms t_i is off by at most 64 * sum |t_i|, the roundings of the terms and of the
division included. The norm's squares are positive: inv is off by 32 + 4 of
itself (the sum's half, eps, root, quotient), y by 2 more, 38, and a scale by 40.
An output in bf16 adds half a step, 2^-8 of the value at most, a code half a code."""
import numpy as np
import pytest
import torch

import combine_topk_ids_02_amd as moe

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24
BF16 = 2.0 ** -8
F64 = torch.float64
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
HS = [8, 24, 32, 504, 512, 520, 2048, 5120, 7168, 8192, 8224, 16384, 16416, 32768]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    moe.lib()


def say(msg):
    print(msg, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def close(got, want, bound, what):
    got = got.to(F64)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / bound)[bad].max()))


def e4m3_bound(v):
    """Half a step of e4m3 at |v| <= 448."""
    low = torch.clamp(v.abs(), min=2.0 ** -6)
    return torch.exp2(torch.floor(torch.log2(low)) - 4)


def check_int8(q, scale, y, y_err, s_err):
    """Codes and scales of rows whose values y (64 bits) the kernel had within
    y_err of themselves."""
    top = y.abs().amax(dim=1)
    close(scale, top / 127.0, s_err * top / 127.0 + 2.0 ** -149, "scale")
    unit = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    off = (q.to(F64) - y * unit[:, None]).abs()
    assert float(off.max()) <= 0.5 + 127 * 2 * y_err, float(off.max())
    assert int(q.to(torch.int32).abs().max()) <= 127
    assert bool((q.to(torch.int32).abs().amax(dim=1)[top > 0] == 127).all())


def check_mxfp8(q, scale, y, y_err):
    T, H = y.shape
    blocks = y.view(T, H // 32, 32)
    top = blocks.abs().amax(dim=2)
    e = scale.to(torch.int64) - 127
    fit = torch.zeros_like(top, dtype=torch.bool)
    for f in (1 - y_err, 1.0, 1 + y_err):  # a top next to a power of two may fall to either side
        want = torch.clamp(torch.floor(torch.log2(torch.clamp(top * f, min=1e-300))) - 8, -127, 127)
        fit |= want == e
    assert bool(fit.all())
    v = (blocks * torch.exp2(-e.to(F64))[..., None]).view(T, H)
    got = q.view(torch.float8_e4m3fn).to(F64)
    want = torch.clamp(v, -448, 448)
    close(got, want, e4m3_bound(want) + y_err * want.abs() + 1e-300, "mxfp8")
    assert bool((torch.signbit(got) == torch.signbit(v))[v != 0].all())


def norm(x, w, eps, res=None, fmt=None, out=True, inv=True):
    """The call, with guard rows behind every output."""
    T, H = x.shape
    d = "cuda"

    def room(dtype, *shape):
        t = torch.empty((shape[0] + 1,) + shape[1:], dtype=dtype, device=d)
        t.view(torch.uint8).fill_(0xA5)
        return t

    o = dict(sum=room(res.dtype, T, H) if res is not None else None,
             out=room(torch.bfloat16, T, H) if out else None,
             inv_rms=room(torch.float32, T) if inv else None, q=None, q_scale=None)
    if fmt == "int8":
        o.update(q=room(torch.int8, T, H), q_scale=room(torch.float32, T))
    elif fmt == "mxfp8":
        o.update(q=room(torch.uint8, T, H), q_scale=room(torch.uint8, T, H // 32))
    moe.norm(x.cuda(), w.cuda(), eps=eps, residual=None if res is None else res.cuda(), fmt=fmt,
             **{k: None if v is None else v[:T] for k, v in o.items()})
    torch.cuda.synchronize()
    for k, v in o.items():
        if v is not None:
            assert bool((v[T:].contiguous().view(torch.uint8) == 0xA5).all()), k
    return {k: None if v is None else v[:T].cpu() for k, v in o.items()}


def check_norm(x, w, eps, res, fmt, o):
    s = x.float()
    if res is not None:
        s = (x.float() + res.float()).to(res.dtype)
        assert torch.equal(o["sum"], s)
    s = s.to(F64)
    inv = 1.0 / torch.sqrt(s.square().mean(dim=1) + eps)
    y = s * inv[:, None] * w.to(F64)
    if o["inv_rms"] is not None:
        close(o["inv_rms"], inv, 36 * ULP * inv, "inv")
    if o["out"] is not None:
        close(o["out"], y, (BF16 + 38 * ULP) * y.abs() + 1e-40, "out")
    if fmt == "int8":
        check_int8(o["q"], o["q_scale"], y, 38 * ULP, 40 * ULP)
    elif fmt == "mxfp8":
        check_mxfp8(o["q"], o["q_scale"], y, 38 * ULP)


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("stream", ["bf16", "f32", None])
def test_norm(H, stream):
    for n, (T, weight, fmt, out) in enumerate([(1, "bf16", None, True), (3, "f32", "int8", True),
                                               (67, "bf16", "int8", False),
                                               (5, "f32", "mxfp8", True),
                                               (66, "bf16", "mxfp8", False)]):
        if fmt == "mxfp8" and H % 32:
            continue
        say(f"norm H={H} T={T} stream={stream} weight={weight} fmt={fmt}")
        g = gen(1000 * H + n)
        x = (randn(g, T, H) * torch.exp(randn(g, T, 1))).to(torch.bfloat16)
        res = None if stream is None else (3 * randn(g, T, H)).to(KINDS[stream])
        w = (1 + 0.2 * randn(g, H)).to(KINDS[weight])
        check_norm(x, w, 1e-6, res, fmt, norm(x, w, 1e-6, res, fmt, out, n != 2))


@pytest.mark.parametrize("fmt", [None, "int8", "mxfp8"])
def test_norm_of_rows_of_every_size(fmt):
    """Zeros, subnormals, the largest values whose squares float32 holds, one value alone."""
    g = gen(3)
    T, H = 9, 256
    x = torch.zeros(T, H)
    x[1] = randn(g, H) * 2.0 ** -130
    x[2] = randn(g, H) * 2.0 ** -60
    x[3] = randn(g, H) * 2.0 ** 55
    x[4, 77] = 1.0
    x[5] = -2.0 ** -133
    x[6] = 448.0
    x[7] = randn(g, H) * torch.exp(4 * randn(g, H))
    x[8] = torch.where(torch.arange(H) % 32 == 5, 1.0, 2.0 ** -12)
    x = x.to(torch.bfloat16)
    w = 1 + 0.2 * randn(g, H)
    w[3], w[64:96] = 0.0, 0.0
    o = norm(x, w, 1e-5, None, fmt)
    check_norm(x, w, 1e-5, None, fmt, o)
    if fmt == "int8":
        assert float(o["q_scale"][0]) == 0 and int(o["q"][0].abs().max()) == 0


def test_norm_where_nothing_is_finite():
    """A NaN or an infinity stays in its row: NaN scales, codes 0 (int8) or NaN."""
    g = gen(4)
    T, H = 4, 5120
    x = randn(g, T, H).to(torch.bfloat16)
    x[1, 4999] = float("nan")
    x[2, 17] = float("inf")
    w = torch.ones(H)
    fine = [0, 3]
    for fmt in (None, "int8", "mxfp8"):
        o = norm(x, w, 1e-6, None, fmt)
        check_norm(x[fine], w, 1e-6, None, fmt, {k: None if v is None else v[fine]
                                                 for k, v in o.items()})
        assert bool(torch.isnan(o["out"][1]).all()) and bool(torch.isnan(o["inv_rms"][1]))
        assert float(o["inv_rms"][2]) == 0.0 and bool(torch.isnan(o["out"][2, 17]))
        if fmt == "int8":
            assert bool(torch.isnan(o["q_scale"][1:3]).all()) and int(o["q"][1:3].abs().max()) == 0
        if fmt == "mxfp8":
            assert bool((o["q_scale"][1] == 255).all())
            assert bool(((o["q"][1] & 0x7F) == 0x7F).all())
            assert int(o["q_scale"][2, 0]) == 255 and int(o["q_scale"][2, 1]) == 0


def test_norm_in_place():
    """sum in the residual's buffer or x's, out in x's: as into buffers of their own."""
    g = gen(5)
    T, H = 33, 7168
    x, res = randn(g, T, H).to(torch.bfloat16), (4 * randn(g, T, H)).to(torch.bfloat16)
    w = (1 + 0.2 * randn(g, H)).to(torch.bfloat16)
    want = norm(x, w, 1e-6, res, "int8")
    for where in ("residual", "x", "both"):
        a, b = x.cuda(), res.cuda()
        out = a if where != "x" else torch.empty_like(a)
        q, s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        total = {"residual": b, "x": a, "both": b}[where]
        moe.norm(a, w.cuda(), residual=b, sum=total, out=out, fmt="int8", q=q, q_scale=s)
        assert torch.equal(total.cpu(), want["sum"]) and torch.equal(out.cpu(), want["out"])
        assert torch.equal(q.cpu(), want["q"]) and torch.equal(s.cpu(), want["q_scale"])
    a, b = x.cuda(), res.cuda()
    out = torch.empty_like(a)
    moe.norm(a, w.cuda(), residual=b, sum=a, out=b)
    assert torch.equal(a.cpu(), want["sum"]) and torch.equal(b.cpu(), want["out"])


def grad_formula(d, h, inv, w, through):
    g = d.to(F64) * w.to(F64)
    u = h.to(F64) * inv.to(F64)[:, None]
    mean = (g * u).mean(dim=1, keepdim=True)
    dh = inv.to(F64)[:, None] * (g - u * mean)
    most = (g * u).abs().mean(dim=1, keepdim=True)
    err = inv.to(F64)[:, None].abs() * (8 * (g.abs() + (u * mean).abs()) + 66 * u.abs() * most)
    if through is not None:
        dh = dh + through.to(F64)
        err = err + 2 * through.to(F64).abs()
    err = ULP * (err + 2 * dh.abs()) + 1e-40
    terms = d.to(F64) * u
    return dh, err, terms.sum(dim=0), terms.abs().sum(dim=0)


def norm_backward(d, h, inv, w, through=None, d_x=True, d_res=True, d_w=True):
    T, H = d.shape

    def room(dtype, *shape):
        t = torch.empty((shape[0] + 16,) + shape[1:], dtype=dtype, device="cuda")
        t.view(torch.uint8).fill_(0xA5)
        return t

    o = dict(d_x=room(torch.bfloat16, T, H) if d_x else None,
             d_residual=room(h.dtype, T, H) if d_res else None,
             d_weight=room(torch.float32, H) if d_w else None)
    n = dict(d_x=T, d_residual=T, d_weight=H)
    need = moe.norm_workspace_bytes(T, H)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs
    moe.norm_backward(d.cuda(), h.cuda(), inv.cuda(), w.cuda(),
                      d_sum=None if through is None else through.cuda(),
                      workspace=ws[:need] if d_w else None,
                      **{k: None if v is None else v[:n[k]] for k, v in o.items()})
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    for k, v in o.items():
        if v is not None:
            assert bool((v[n[k]:].contiguous().view(torch.uint8) == 0xA5).all()), k
    return {k: None if v is None else v[:n[k]].cpu() for k, v in o.items()}


def check_grad(d, h, inv, w, through, o):
    dh, err, dw, terms = grad_formula(d, h, inv, w, through)
    if o["d_x"] is not None:
        close(o["d_x"], dh, err + BF16 * dh.abs(), "d_x")
    if o["d_residual"] is not None:
        half = BF16 if h.dtype == torch.bfloat16 else 0.0
        close(o["d_residual"], dh, err + half * dh.abs(), "d_residual")
    if o["d_weight"] is not None:
        # a term is rounded once with its u and once when it is added; a thread adds at
        # most ceil(T / 512) of them, or one of each 16 where a workgroup has several
        # rows, and then up to 16 threads' sums are added in float32; the workgroups'
        # in 64 bits
        adds = -(-d.shape[0] // 512) + 16
        close(o["d_weight"], dw, ULP * ((adds + 1) * terms + dw.abs()) + 1e-40, "d_weight")


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_norm_backward(H, stream):
    for n, (T, weight, through) in enumerate([(1, "bf16", False), (3, "f32", True),
                                              (70, "bf16", True),
                                              (1031 if H <= 5120 else 515, "f32", False)]):
        say(f"norm_backward H={H} T={T} stream={stream} weight={weight} through={through}")
        g = gen(77 * H + n)
        h = (randn(g, T, H) * torch.exp(randn(g, T, 1))).to(KINDS[stream])
        inv = (1.0 / torch.sqrt(h.to(F64).square().mean(dim=1) + 1e-6)).float()
        w = (1 + 0.2 * randn(g, H)).to(KINDS[weight])
        d = randn(g, T, H).to(torch.bfloat16)
        t = randn(g, T, H).to(KINDS[stream]) if through else None
        check_grad(d, h, inv, w, t, norm_backward(d, h, inv, w, t, n != 1, n != 2, n != 0))


def test_norm_backward_against_differences():
    """The gradient of sum(d_out * y) + sum(d_sum * h) by central differences of
    the formula in 64 bits."""
    g = gen(8)
    T, H = 4, 48
    h = randn(g, T, H)
    d, t = randn(g, T, H).to(torch.bfloat16), randn(g, T, H)
    w = 1 + 0.2 * randn(g, H)

    def loss(hh, ww):
        y = hh / torch.sqrt(hh.square().mean(dim=1, keepdim=True) + 1e-6) * ww
        return ((d.to(F64) * y).sum() + (t.to(F64) * hh).sum()).item()

    inv = (1.0 / torch.sqrt(h.to(F64).square().mean(dim=1) + 1e-6)).float()
    o = norm_backward(d, h, inv, w, t)
    h64, w64 = h.to(F64), w.to(F64)
    step = 1e-5
    for r, c in [(0, 0), (1, 7), (2, 33), (3, 47), (3, 8)]:
        e = torch.zeros(T, H, dtype=F64)
        e[r, c] = step
        slope = (loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * step)
        assert abs(slope - float(o["d_residual"][r, c])) < 1e-5  # step^2 and 64-bit noise / step
        f = torch.zeros(H, dtype=F64)
        f[c] = step
        slope = (loss(h64, w64 + f) - loss(h64, w64 - f)) / (2 * step)
        assert abs(slope - float(o["d_weight"][c])) < 1e-5


def test_norm_backward_in_place_and_empty():
    g = gen(9)
    T, H = 37, 5120
    h, t = randn(g, T, H), randn(g, T, H)
    inv = (1.0 / torch.sqrt(h.to(F64).square().mean(dim=1) + 1e-6)).float()
    w, d = 1 + 0.2 * randn(g, H), randn(g, T, H).to(torch.bfloat16)
    want = norm_backward(d, h, inv, w, t)
    a, b = d.cuda(), t.cuda()
    moe.norm_backward(a, h.cuda(), inv.cuda(), w.cuda(), d_sum=b, d_x=a, d_residual=b)
    assert torch.equal(a.cpu(), want["d_x"]) and torch.equal(b.cpu(), want["d_residual"])
    o = norm_backward(d[:0], h[:0], inv[:0], w)
    assert bool((o["d_weight"] == 0).all())
    o = norm(h[:0].to(torch.bfloat16), w, 1e-6, h[:0], "int8")
    assert o["q"].shape == (0, H)


def quantise(rows, pair_row=None):
    cap = rows.shape[0]
    H = rows.shape[1]
    q = torch.full((cap + 1, H), 0x55, dtype=torch.int8, device="cuda")
    s = torch.full((cap + 1,), -7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.quantise_rows(rows.cuda(), q[:cap], s[:cap], err=err,
                      pair_row=None if pair_row is None else pair_row.cuda())
    torch.cuda.synchronize()
    assert bool((q[cap:] == 0x55).all()) and bool((s[cap:] == -7.0).all())
    return q[:cap].cpu(), s[:cap].cpu(), int(err.item())


@pytest.mark.parametrize("H", [8, 40, 512, 1000, 1024, 2048, 2056, 5120, 8192, 8200, 16384, 16392,
                               40000, 65536])
def test_quantise_rows(H):
    for T in (1, 2, 7, 70):
        say(f"quantise_rows H={H} T={T}")
        g = gen(13 * H + T)
        rows = (randn(g, T, H) * torch.exp(3 * randn(g, T, 1))).to(torch.bfloat16)
        q, s, err = quantise(rows)
        assert err == 0
        check_int8(q, s, rows.to(F64), 2 * ULP, 2 * ULP)  # reciprocal, factor, product


def test_quantise_rows_of_every_size():
    g = gen(21)
    H = 2048
    rows = torch.zeros(10, H)
    rows[1] = randn(g, H) * 2.0 ** -128
    rows[2] = 2.0 ** -133
    rows[3] = randn(g, H) * 2.0 ** 124
    rows[4, 3] = -3.3e38
    rows[5] = float("nan")
    rows[6, 2047] = float("-inf")
    rows[7, 8] = float("nan")
    rows[8] = randn(g, H) * 2.0 ** -66
    rows[9] = -1.0
    rows = rows.to(torch.bfloat16)
    for wide in (1, 3):  # a row per wave, and a row per workgroup
        r = rows.repeat(1, wide)
        q, s, _ = quantise(r)
        fine = [0, 1, 2, 3, 4, 8, 9]
        check_int8(q[fine], s[fine], r[fine].to(F64), 3 * ULP, 3 * ULP)
        assert bool(torch.isnan(s[5:8]).all()) and int(q[5:8].abs().max()) == 0
        assert float(s[0]) == 0.0 and int(q[0].abs().max()) == 0
        assert int(q[9].min()) == int(q[9].max()) == -127


@pytest.mark.parametrize("H", [512, 4096])
def test_quantise_rows_of_pairs(H):
    """Only the rows that pair_row names; -1 is skipped, rows past the buffer are flagged."""
    g = gen(22)
    T, k, cap = 29, 3, 150
    rows = randn(g, cap, H).to(torch.bfloat16)
    at = torch.randperm(cap, generator=g)[:T * k].to(torch.int32).view(T, k)
    at[4, 1], at[20, 0] = -1, -1
    q, s, err = quantise(rows, at)
    assert err == 0
    live = torch.zeros(cap, dtype=torch.bool)
    live[at[at >= 0].long()] = True
    check_int8(q[live], s[live], rows[live].to(F64), 2 * ULP, 2 * ULP)
    assert bool((q[~live] == 0x55).all()) and bool((s[~live] == -7.0).all())
    at[0, 0], at[5, 2] = cap, 2 ** 31 - 1
    q2, s2, err = quantise(rows, at)
    assert err == moe.ERRBIT_EXPERT_CAP
    kept = torch.zeros(cap, dtype=torch.bool)
    kept[at[(at >= 0) & (at < cap)].long()] = True
    assert torch.equal(q2[kept], q[kept]) and bool((q2[~kept] == 0x55).all())


def test_rows_far_into_a_buffer():
    """Rows behind the 2^31st value: offsets of 64 bits."""
    H, cap = 65536, 33000
    rows = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
    g = gen(23)
    some = randn(g, 2, H).to(torch.bfloat16)
    rows[[32766, 32999]] = some.cuda()
    q = torch.zeros(cap, H, dtype=torch.int8, device="cuda")
    s = torch.zeros(cap, device="cuda")
    at = torch.tensor([[32766, 32999]], dtype=torch.int32, device="cuda")
    moe.quantise_rows(rows, q, s, pair_row=at)
    check_int8(q[[32766, 32999]].cpu(), s[[32766, 32999]].cpu(), some.to(F64), 2 * ULP, 2 * ULP)
    assert float(s[:32766].abs().max()) == 0
    del rows, q
    T, H = 65540, 32768
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-1] = some[0, :H].cuda()
    x[0] = some[1, :H].cuda()
    w, out = torch.ones(H, device="cuda"), torch.empty_like(x)
    moe.norm(x, w, out=out)
    pick = [0, T - 1]
    o = dict(sum=None, out=out[pick].cpu(), inv_rms=None)
    check_norm(x[pick].cpu(), w.cpu(), 1e-6, None, None, o)
    assert float(out[1:-1].abs().max()) == 0


def test_norm_and_gradient_in_a_graph_and_on_a_stream():
    """Captured once on another stream and replayed with new inputs, with eager
    work between the replays: as the eager calls."""
    g = gen(30)
    T, H = 130, 5120
    x, d = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(
        T, H, dtype=torch.bfloat16, device="cuda")
    res, w = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda")
    q2 = torch.empty(T, H, dtype=torch.int8, device="cuda")
    s2 = torch.empty(T, device="cuda")

    def fill():
        x.copy_(randn(g, T, H))
        d.copy_(randn(g, T, H))
        res.copy_(randn(g, T, H))
        w.copy_(1 + 0.2 * randn(g, H))

    def buffers():
        f32 = dict(device="cuda")
        return dict(sum=torch.empty(T, H, **f32), out=torch.empty_like(x),
                    inv=torch.empty(T, **f32), q=torch.empty_like(q2), s=torch.empty(T, **f32),
                    dx=torch.empty_like(x), dr=torch.empty(T, H, **f32),
                    dw=torch.empty(H, **f32), q2=torch.empty_like(q2), s2=torch.empty(T, **f32),
                    ws=torch.empty(moe.norm_workspace_bytes(T, H), dtype=torch.uint8, **f32))

    def step(b):
        moe.norm(x, w, residual=res, sum=b["sum"], out=b["out"], fmt="int8", q=b["q"],
                 q_scale=b["s"], inv_rms=b["inv"])
        moe.norm_backward(d, b["sum"], b["inv"], w, d_sum=res, d_x=b["dx"], d_residual=b["dr"],
                          d_weight=b["dw"], workspace=b["ws"])
        moe.quantise_rows(b["out"], b["q2"], b["s2"])

    fill()
    b, e = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(b)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(b)
    for n in range(4):
        fill()
        for t in b.values():
            t.zero_()
        graph.replay()
        if n % 2:
            torch.cuda.synchronize()
        step(e)
        torch.cuda.synchronize()
        for key in b:
            if key != "ws":
                assert torch.equal(b[key], e[key]), (n, key)
