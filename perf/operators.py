"""Cases of the router, its balance loss and the expert products with 4-bit
weights: inputs, the operators in elementary torch operations (`own` false) or
through the package (`own` true), and their values in 64 bits.

An operator is one of
  route      router logits [T, E] -> the k experts of each token and their weights
  grad       the gradient of the router's logits, from the weights' gradient,
             from the balance loss's, or from both at once
  balance    the balance loss of each sequence, with the pairs of each expert
  product    expert-grouped rows times their experts' 4-bit weights
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GROUP = {"mxfp4": 32, "nvfp4": 16}  # values that share one scale byte
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token of one request, the router of a decode step without a batch
        dict(name="route_token", op="route", T=1, E=256, k=8, dtype="bf16", scoring="sigmoid",
             renorm=True, scale=2.5, bias=True, groups=8, top_groups=4, masked=0),
        # the decode step of the benchmark: 64 requests, 384 experts, top-6
        dict(name="route_decode", op="route", T=64, E=384, k=6, dtype="f32", scoring="softmax",
             renorm=True, scale=1.0, bias=False, groups=1, top_groups=1, masked=0),
        # its prefill chunk, not quite full, the last tokens being padding
        dict(name="route_prefill", op="route", T=4093, E=384, k=6, dtype="f32",
             scoring="softmax", renorm=True, scale=1.0, bias=False, groups=1, top_groups=1,
             masked=119),
        # the large chunk with group-limited choice by biased sigmoid scores
        dict(name="route_chunk", op="route", T=16384, E=256, k=8, dtype="f32",
             scoring="sigmoid", renorm=True, scale=2.5, bias=True, groups=8, top_groups=4,
             masked=0),
        # a training step's whole gradient of the router's logits
        dict(name="grad_step", op="grad", T=8192, E=256, k=8, dtype="bf16", scoring="sigmoid",
             renorm=True, scale=2.5, weights=True, S=1, masked=57),
        # the balance loss alone, over ragged sequences
        dict(name="grad_balance", op="grad", T=16384, E=256, k=8, dtype="f32",
             scoring="softmax", renorm=True, scale=1.0, weights=False, S=13, masked=0),
        # one loss over the whole batch
        dict(name="balance_batch", op="balance", T=4096, E=384, k=6, dtype="f32",
             scoring="softmax", S=1, masked=0),
        # one loss for each of 13 packed sequences, padding behind them
        dict(name="balance_sequences", op="balance", T=16384, E=256, k=8, dtype="bf16",
             scoring="sigmoid", S=13, masked=200),
        # one token's first expert product (gate and up, joined by SwiGLU) on
        # the 48 experts of one of 8 ranks
        dict(name="product_token", op="product", T=1, k=6, E=48, K=5120, N=4096, fmt="mxfp4",
             act="swiglu", factor=False, align=1, block=0),
        # the first product of a decode step, as many pairs as 64 requests make
        dict(name="product_decode", op="product", T=64, k=6, E=48, K=5120, N=4096, fmt="nvfp4",
             act="swiglu", factor=True, align=1, block=0),
        # and the second, back to the hidden size
        dict(name="product_down", op="product", T=64, k=6, E=48, K=2048, N=5120, fmt="mxfp4",
             act="none", factor=False, align=1, block=0),
        # the largest decode-sized batch, in fixed blocks of rows per expert
        dict(name="product_batch", op="product", T=256, k=8, E=32, K=7168, N=4096, fmt="mxfp4",
             act="swiglu", factor=False, align=1, block=256),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "grad", "balance", "product", "product"])
    if op == "product":
        while True:
            act = rng.choice(["none", "swiglu"])
            N = rng.randint(256, 5120)
            c = dict(op=op, T=_log(rng, 1, 256), k=rng.randint(1, 8), E=_log(rng, 8, 64),
                     K=32 * rng.randint(16, 224), N=N - N % 2 if act == "swiglu" else N,
                     fmt=rng.choice(["mxfp4", "nvfp4"]), act=act, factor=rng.random() < 0.5,
                     align=1, block=0)
            shape = rng.choice(["runs", "runs", "padded", "blocks"])
            if shape == "padded":
                c["align"] = rng.choice([16, 64, 128])
            elif shape == "blocks":
                c["block"] = c["T"]
            if c["E"] * c["N"] * c["K"] <= 32 * 4096 * 7168:
                return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 16384), E=_log(rng, 8, 512), k=rng.randint(1, 8),
                 dtype=rng.choice(["f32", "bf16", "f16"]),
                 scoring=rng.choice(["softmax", "sigmoid"]))
        c["masked"] = rng.choice([0, c["T"] // 9])
        if c["T"] * c["E"] > 16384 * 256:
            continue
        if op == "balance":
            c["S"] = _log(rng, 1, 24)
            return c
        c["renorm"] = rng.random() < 0.7
        c["scale"] = rng.choice([1.0, 2.5])
        if op == "grad":
            c["weights"] = rng.random() < 0.7
            c["S"] = rng.randint(0 if c["weights"] else 1, 20)
            return c
        c.update(bias=False, groups=1, top_groups=1)
        if c["scoring"] == "sigmoid":
            c["bias"] = rng.random() < 0.7
            ways = [g for g in (1, 2, 4, 8) if c["E"] % g == 0]
            c["groups"] = rng.choice(ways)
            c["top_groups"] = rng.randint(max(1, c["groups"] // 2), c["groups"])
        return c


# ---------------------------------------------------------------------------
# Inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _logits(c, g):
    """N(0, 1) with a popularity of each expert, as a router's come out."""
    z = torch.randn(c["T"], c["E"], device="cuda", generator=g)
    z += 0.5 * torch.randn(c["E"], device="cuda", generator=g)
    return z.to(DTYPES[c["dtype"]])


def _sequences(c, g):
    """Offsets of S packed sequences of uneven lengths; the masked tokens lie
    behind the last one."""
    S, n = c["S"], c["T"] - c["masked"]
    cuts = torch.randint(0, n + 1, (S - 1,), device="cuda", generator=g).sort().values
    ends = torch.tensor([n], device="cuda")
    return torch.cat([ends * 0, cuts, ends]).to(torch.int32)


def _chosen(c, z, g):
    """Ids as a router gives them: the k best of perturbed logits, the masked
    tokens with none."""
    noise = 0.1 * torch.randn(z.shape, device="cuda", generator=g)
    ids = (z.float() + noise).topk(c["k"], dim=1).indices.to(torch.int32)
    if c["masked"]:
        ids[c["T"] - c["masked"]:] = -1
    return ids.contiguous()


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _f32(*shape):
    return torch.zeros(shape, dtype=torch.float32, device="cuda")


def prepare(case, seed):
    c, g = case, _generator(seed)
    if c["op"] == "product":
        return _prepare_product(c, g)
    s = dict(case=c, logits=_logits(c, g))
    if own:
        import combine_topk_ids_02_amd as moe
        s["router"] = moe.Router(scoring=c["scoring"], renorm=c.get("renorm", True),
                                 scale=c.get("scale", 1.0), groups=c.get("groups", 1),
                                 top_groups=c.get("top_groups", 1))
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "route":
        s["bias"] = 0.1 * torch.randn(E, device="cuda", generator=g) if c["bias"] else None
        s["mask"] = None
        if c["masked"]:
            s["mask"] = torch.arange(T, device="cuda") < T - c["masked"]
        s["ids"], s["weights"] = _i32(T, k), _f32(T, k)
        return s
    s["ids"] = _chosen(c, s["logits"], g)
    s["offsets"] = _sequences(c, g) if c["S"] > 0 else None
    if c["op"] == "balance":
        S = c["S"]
        s.update(loss=_f32(S), counts=_i32(S, E), tokens=_i32(S), mean=_f32(S, E))
        if own:
            need = moe.balance_workspace_bytes(T, E, k, S)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return s
    s["d_weights"] = None
    if c["weights"]:
        s["d_weights"] = torch.randn(T, k, device="cuda", generator=g) / 64
    if c["S"] > 0:
        s["counts"], s["tokens"] = _count(s["ids"], s["offsets"], E)
        s["d_loss"] = 0.01 * (1 + torch.rand(c["S"], device="cuda", generator=g))
    s["d_logits"] = torch.zeros_like(s["logits"])
    return s


def _prepare_product(c, g):
    T, k, E, K, N = c["T"], c["k"], c["E"], c["K"], c["N"]
    # routing with popular and rare experts
    z = torch.randn(T, E, device="cuda", generator=g)
    z += 0.5 * torch.randn(E, device="cuda", generator=g)
    ids = z.topk(k, dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    if c["block"] > 0:
        offsets = torch.arange(E + 1, device="cuda") * c["block"]
        cap = E * c["block"]
    else:
        runs = (counts + c["align"] - 1) // c["align"] * c["align"]
        offsets = torch.cat([runs.new_zeros(1), runs.cumsum(0)])
        cap = T * k + E * (c["align"] - 1)
    rows = torch.randn(cap, K, device="cuda", generator=g).to(torch.bfloat16)
    # codes distributed as a quantised normal tensor's: 256 quantiles of
    # N(0, 2) rounded to the e2m1 grid, one drawn for each nibble
    q = 2.0 * torch.special.ndtri((torch.arange(256, device="cuda") + 0.5) / 256)
    grid = torch.tensor(E2M1, device="cuda")
    code = (q[:, None] - grid[None, :]).abs().argmin(dim=1).to(torch.uint8)
    pair = (code[:, None] | (code[None, :] << 4)).reshape(-1)
    w_q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    for e in range(E):
        two = torch.randint(0, 65536, (N, K // 2), device="cuda", generator=g, dtype=torch.int32)
        w_q[e] = pair[two]
    blk = GROUP[c["fmt"]]
    if c["fmt"] == "mxfp4":  # 2^-8 .. 2^-5: weights of about 1 / sqrt(K)
        w_s = torch.randint(119, 123, (E, N, K // blk), device="cuda", generator=g,
                            dtype=torch.uint8)
    else:  # e4m3 bytes of 2^-7 .. 2^-4
        w_s = torch.randint(5, 25, (E, N, K // blk), device="cuda", generator=g,
                            dtype=torch.uint8)
    factor = None
    if c["factor"]:
        factor = 0.5 + torch.rand(E, device="cuda", generator=g)
    wide = N // 2 if c["act"] == "swiglu" else N
    return dict(case=c, rows=rows, counts=counts.to(torch.int32), offsets=offsets.to(torch.int32),
                w_q=w_q, w_scale=w_s, factor=factor,
                out=torch.zeros(cap, wide, dtype=torch.bfloat16, device="cuda"))


# ---------------------------------------------------------------------------
# One pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import combine_topk_ids_02_amd as moe
    c = s["case"]
    if c["op"] == "route":
        moe.route(s["logits"], c["k"], s["router"], s["ids"], s["weights"], bias=s["bias"],
                  token_mask=s["mask"])
        return s["ids"], s["weights"]
    if c["op"] == "balance":
        moe.balance_loss(s["logits"], s["ids"], s["router"], s["loss"], s["counts"], s["tokens"],
                         s["mean"], seq_offsets=s["offsets"] if c["S"] > 1 else None,
                         workspace=s["workspace"])
        return s["loss"], s["counts"], s["tokens"], s["mean"]
    if c["op"] == "grad":
        balance = None
        if c["S"] > 0:
            balance = (s["d_loss"], s["counts"], s["tokens"], s["offsets"])
        moe.route_backward(s["logits"], s["ids"], s["router"], s["d_logits"],
                           d_weights=s["d_weights"], balance=balance)
        return s["d_logits"]
    moe.expert_product(c["fmt"], s["rows"], s["counts"], s["offsets"], c["T"], c["k"], s["w_q"],
                       s["w_scale"], s["out"], act=c["act"], factor=s["factor"])
    return s["out"]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _plain_route(c, s["logits"], s["bias"], s["mask"])
    if c["op"] == "balance":
        return _plain_balance(c, s["logits"], s["ids"], s["offsets"])
    if c["op"] == "grad":
        return _plain_grad(c, s)
    return _plain_product(c, s)


def _plain_route(c, logits, bias, mask):
    T, E, k = c["T"], c["E"], c["k"]
    z = logits.float()
    low = torch.full_like(z, -math.inf)
    if c["scoring"] == "softmax" or (bias is None and c["groups"] == 1):
        key = z
    else:  # the score as float32, from 64 bits: two keys may differ in its last bit
        key = (1.0 / (1.0 + torch.exp(-z.double()))).float()
        key = key if bias is None else key + bias
        key = torch.where(z == -math.inf, low, key)
    fine = ((z < math.inf) & (key < math.inf)).all(dim=1, keepdim=True)
    if mask is not None:
        fine = fine & mask[:, None]
    if c["groups"] > 1:
        G = c["groups"]
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values
        total = best[..., 0]
        if E // G > 1:
            total = torch.where(best[..., 1] > -math.inf, total + best[..., 1], total)
        order = total.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device)
        keep.scatter_(1, order[:, :c["top_groups"]], True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, low)
    found = key.sort(dim=1, descending=True, stable=True)
    ok = (found.values[:, :k] > -math.inf) & fine
    ids = found.indices[:, :k]
    zc = torch.gather(z, 1, ids)
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-zc))
    else:
        top = z.amax(dim=1, keepdim=True)
        score = torch.exp(zc - top)
        if not c["renorm"]:
            score = score / torch.exp(z - top).sum(dim=1, keepdim=True)
    score = torch.where(ok, score, torch.zeros_like(score))
    if c["renorm"]:
        total = score.sum(dim=1, keepdim=True)
        score = score / torch.where(total > 0, total, torch.ones_like(total))
    ids = torch.where(ok, ids, torch.full_like(ids, -1)).to(torch.int32)
    return ids, score * c["scale"]


def _segments(T, offsets):
    """Each token's sequence, and whether it lies in one."""
    t = torch.arange(T, device=offsets.device, dtype=torch.int32)
    seq = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    inside = (t >= offsets[0]) & (t < offsets[-1])
    return seq.clamp(max=offsets.numel() - 2), inside


def _count(ids, offsets, E):
    """Pairs per (sequence, expert) and tokens with an expert per sequence."""
    S = offsets.numel() - 1
    seq, inside = _segments(ids.shape[0], offsets)
    ok = (ids >= 0) & inside[:, None]
    cell = torch.where(ok, seq[:, None] * E + ids, S * E).reshape(-1)
    counts = torch.bincount(cell, minlength=S * E + 1)[:S * E].view(S, E)
    tokens = torch.bincount(torch.where(ok.any(dim=1), seq, S), minlength=S + 1)[:S]
    return counts.to(torch.int32), tokens.to(torch.int32)


def _shares(c, z):
    """The scores of every token scaled to a sum of one."""
    if c["scoring"] == "softmax":
        p = torch.exp(z - z.amax(dim=1, keepdim=True))
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
    return p / p.sum(dim=1, keepdim=True)


def _plain_balance(c, logits, ids, offsets):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    counts, tokens = _count(ids, offsets, E)
    seq, inside = _segments(T, offsets)
    used = (ids >= 0).any(dim=1) & inside
    share = _shares(c, logits.float()).double() * used[:, None]
    member = torch.arange(S, device=logits.device)[:, None] == seq[None, :]
    total = torch.matmul(member.double(), share)
    mean = total / tokens.clamp(min=1)[:, None]
    loss = (counts * mean).sum(dim=1) * (E / k) / tokens.clamp(min=1)
    return loss.float(), counts, tokens, mean.float()


def _plain_grad(c, s):
    z, ids = s["logits"].float(), s["ids"].long()
    T, E, k = c["T"], c["E"], c["k"]
    ok = ids >= 0
    at = ids.clamp(min=0)
    total = torch.zeros_like(z)
    slope = torch.ones_like(z)
    if c["scoring"] == "sigmoid":
        slope = 1.0 / (1.0 + torch.exp(z))
    if s["d_weights"] is not None:
        g = torch.where(ok, s["d_weights"], torch.zeros_like(s["d_weights"])) * c["scale"]
        zc = torch.gather(z, 1, at)
        if c["renorm"]:
            if c["scoring"] == "softmax":
                top = torch.where(ok, zc, torch.full_like(zc, -math.inf)).amax(1, keepdim=True)
                q = torch.exp(zc - torch.where(ok, top, zc))
            else:
                q = 1.0 / (1.0 + torch.exp(-zc))
            q = torch.where(ok, q, torch.zeros_like(q))
            q = q / q.sum(dim=1, keepdim=True).clamp(min=1e-30)
            part = q * (g - (q * g).sum(dim=1, keepdim=True))
            part = part * torch.gather(slope, 1, at)
            total.scatter_add_(1, at, part)
        elif c["scoring"] == "softmax":
            p = _shares(c, z)
            up = torch.zeros_like(z).scatter_add_(1, at, g)
            total += p * (up - (p * up).sum(dim=1, keepdim=True))
        else:
            sig = 1.0 / (1.0 + torch.exp(-zc))
            total.scatter_add_(1, at, g * sig * torch.gather(slope, 1, at))
    if c["S"] > 0:
        seq, inside = _segments(T, s["offsets"])
        tokens = s["tokens"].clamp(min=1).double()
        rate = (s["d_loss"].double() * E / (k * tokens * tokens))[:, None] * s["counts"]
        # subtracting one number from a row's rates changes no gradient
        rate = (rate - rate.mean(dim=1, keepdim=True)).float()[seq]
        p = _shares(c, z)
        part = p * slope * (rate - (p * rate).sum(dim=1, keepdim=True))
        total += torch.where((ok.any(dim=1) & inside)[:, None], part, torch.zeros_like(part))
    return total.to(s["logits"].dtype)


def _weights_plain(c, w_q, w_scale):
    pairs = torch.tensor(E2M1, device=w_q.device)
    pairs = torch.stack([pairs.repeat(16), pairs.repeat_interleave(16)], dim=1)
    E, N, half = w_q.shape
    w = pairs[w_q.int()].view(E, N, w_scale.shape[2], GROUP[c["fmt"]])
    if c["fmt"] == "mxfp4":
        scale = (w_scale.int() << 23).view(torch.float32)
    else:
        scale = w_scale.view(torch.float8_e4m3fn).float()
    return (w * scale[..., None]).view(E, N, 2 * half)


def _plain_product(c, s):
    E, K, N = c["E"], c["K"], c["N"]
    most = min(c["T"], c["block"]) if c["block"] > 0 else c["T"]  # rows of one expert
    cap = s["rows"].shape[0]
    row = torch.arange(cap, device="cuda", dtype=torch.int32)
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True).clamp(max=E - 1)
    place = row - s["offsets"][expert]
    live = place < s["counts"][expert]
    spot = torch.where(live, expert * most + place, E * most)
    x = torch.zeros(E * most + 1, K, device="cuda")
    x[spot] = s["rows"].float()
    x = x[:E * most].view(E, most, K).transpose(1, 2).contiguous()
    y = torch.bmm(_weights_plain(c, s["w_q"], s["w_scale"]), x)
    if s["factor"] is not None:
        y = y * s["factor"][:, None, None]
    if c["act"] == "swiglu":
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    y = y.transpose(1, 2).reshape(E * most, -1).to(torch.bfloat16)
    y = torch.cat([y, y.new_zeros(1, y.shape[1])])
    return y[spot]


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c = case
    if c["op"] == "product":
        pairs, E, K, N = c["T"] * c["k"], c["E"], c["K"], c["N"]
        # the experts that uniform routing reaches
        live = E * (1.0 - (1.0 - min(1.0, c["k"] / E)) ** c["T"])
        wide = N // 2 if c["act"] == "swiglu" else N
        per = N * K * (0.5 + 1.0 / GROUP[c["fmt"]])
        return {"bytes": live * per + pairs * 2 * (K + wide), "flops": 2 * pairs * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "route":
        return {"bytes": T * E * size + 8 * T * k, "flops": 4 * T * E}
    if c["op"] == "balance":
        return {"bytes": T * E * size + 4 * T * k + 8 * c["S"] * E, "flops": 5 * T * E}
    return {"bytes": 2 * T * E * size + 4 * T * k * (2 if c["weights"] else 1)
            + 4 * c["S"] * E, "flops": 8 * T * E}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, on the host (the products on the GPU)


def _sig(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def _host(t):
    return t.to(torch.float64).cpu().numpy()


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "product":
        return _exact_product(c, s)
    z, ids = _host(s["logits"]), s["ids"].cpu().numpy()
    sig = _sig(z)
    if c["scoring"] == "softmax":
        share = np.exp(z - z.max(axis=1, keepdims=True))
        inner = np.ones_like(z)
    else:
        share, inner = sig, 1.0 - sig
    share = share / share.sum(axis=1, keepdims=True)
    bounds = s["offsets"].cpu().numpy() if c["S"] > 0 else [0]
    if c["op"] == "balance":
        return _exact_balance(c, share, ids, bounds)
    T, E, k = c["T"], c["E"], c["k"]
    d = np.zeros_like(z)
    if c["weights"]:
        g = _host(s["d_weights"]) * c["scale"]
        chosen = np.zeros((T, E))
        up = np.zeros((T, E))
        for j in range(k):
            t = np.nonzero(ids[:, j] >= 0)[0]
            chosen[t, ids[t, j]] += 1.0
            up[t, ids[t, j]] += g[t, j]
        score = share if c["scoring"] == "softmax" else sig
        if c["renorm"]:
            q = score * chosen
            q = q / np.where(q.sum(1, keepdims=True) > 0, q.sum(1, keepdims=True), 1.0)
            d += inner * q * (up - (q * up).sum(axis=1, keepdims=True))
        elif c["scoring"] == "softmax":
            d += share * (up - (share * up).sum(axis=1, keepdims=True))
        else:
            d += up * sig * inner
    weight = s["d_loss"].cpu().numpy().astype(np.float64) if c["S"] > 0 else None
    for i in range(c["S"]):
        a, b = int(bounds[i]), int(bounds[i + 1])
        live = (ids[a:b] >= 0).any(axis=1)
        n = live.sum()
        if n == 0:
            continue
        count = np.bincount(ids[a:b][ids[a:b] >= 0], minlength=E)
        rate = weight[i] * E / (k * float(n) ** 2) * count
        p = share[a:b]
        part = p * inner[a:b] * (rate[None, :] - (p @ rate)[:, None])
        d[a:b] += part * live[:, None]
    return d


def _exact_route(c, s):
    z = _host(s["logits"])
    T, E, k = c["T"], c["E"], c["k"]
    key = z.astype(np.float32)
    if c["bias"] or c["groups"] > 1:
        key = _sig(z).astype(np.float32)
        if c["bias"]:
            key = key + s["bias"].cpu().numpy()
    key = key.astype(np.float64)
    if c["groups"] > 1:
        G, m = c["groups"], E // c["groups"]
        cells = key.astype(np.float32).reshape(T, G, m)
        two = -np.sort(-cells, axis=2)[:, :, :2]
        total = two[..., 0] + two[..., 1] if m > 1 else two[..., 0]
        order = np.argsort(-total, axis=1, kind="stable")
        for t in range(T):
            for gi in order[t, c["top_groups"]:]:
                key[t, gi * m:(gi + 1) * m] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    rows = np.arange(T)[:, None]
    live = key[rows, ids] > -np.inf
    live &= (np.arange(T) < T - c["masked"])[:, None]
    if c["scoring"] == "sigmoid":
        score = _sig(z)[rows, ids]
    else:
        e = np.exp(z - z.max(axis=1, keepdims=True))
        score = (e / e.sum(axis=1, keepdims=True))[rows, ids]
    score = score * live
    if c["renorm"]:
        total = score.sum(axis=1, keepdims=True)
        score = score / np.where(total > 0, total, 1.0)
    return np.where(live, ids, -1).astype(np.int32), score * c["scale"]


def _exact_balance(c, share, ids, bounds):
    E, k, S = c["E"], c["k"], c["S"]
    loss, mean = np.zeros(S), np.zeros((S, E))
    counts, tokens = np.zeros((S, E), np.int32), np.zeros(S, np.int32)
    for i in range(S):
        a, b = int(bounds[i]), int(bounds[i + 1])
        live = (ids[a:b] >= 0).any(axis=1)
        tokens[i] = live.sum()
        if tokens[i] == 0:
            continue
        counts[i] = np.bincount(ids[a:b][ids[a:b] >= 0], minlength=E)
        mean[i] = share[a:b][live].sum(axis=0) / tokens[i]
        loss[i] = E / (k * float(tokens[i])) * (counts[i] * mean[i]).sum()
    return loss, counts, tokens, mean


def _exact_product(c, s):
    N, K, blk = c["N"], c["K"], GROUP[c["fmt"]]
    counts, offsets = s["counts"].tolist(), s["offsets"].tolist()
    value = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        if counts[e] == 0:
            continue
        a = offsets[e]
        b = a + counts[e]
        byte = s["w_q"][e]
        w = torch.empty(N, K, dtype=torch.float64, device="cuda")
        w[:, 0::2] = value[(byte & 15).long()]
        w[:, 1::2] = value[(byte >> 4).long()]
        code = s["w_scale"][e].double()
        if c["fmt"] == "mxfp4":
            scale = torch.exp2(code - 127.0)
        else:  # exponent 4 bits with bias 7, mantissa 3 bits
            top, low = torch.floor(code / 8), torch.remainder(code, 8)
            scale = torch.where(top > 0, (8 + low) * torch.exp2(top - 10.0), low * 2.0 ** -9)
        w = (w.view(N, K // blk, blk) * scale[..., None]).view(N, K)
        y = s["rows"][a:b].double() @ w.t().contiguous()
        if s["factor"] is not None:
            y = y * s["factor"][e].double()
        if c["act"] == "swiglu":
            gate, up = y[:, :N // 2], y[:, N // 2:]
            y = gate / (1.0 + torch.exp(-gate)) * up
        out[a:b] = y
    return out
