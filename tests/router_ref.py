"""The router, its gradient, the balance loss and the 4-bit expert products in
64 bits (numpy), straight from their formulas and apart from the kernels: what
the tests compare with, and the sizes of the terms their tolerances count."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0,
                 -4.0, -6.0])
ULP = 2.0 ** -24  # half a step of float32, relative


def sigmoid(z):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))),
                        np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


def keys(z, scoring, bias, groups):
    z = np.asarray(z, np.float64)
    if scoring == "softmax" or (bias is None and groups == 1):
        return z.copy()
    with np.errstate(invalid="ignore"):
        key = sigmoid(z).astype(np.float32)
        if bias is not None:
            key = key + np.asarray(bias, np.float32)
    key = key.astype(np.float64)
    key[z == -np.inf] = -np.inf
    return key


def choose(z, k, scoring, bias=None, groups=1, top_groups=1, mask=None):
    """ids [T, k] and whether any token had a NaN or +infinite logit or key."""
    T, E = z.shape
    ids = np.full((T, k), -1, np.int64)
    flagged = False
    key = keys(z, scoring, bias, groups)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        if not (np.all(z[t] < np.inf) and np.all(key[t] < np.inf)):
            flagged = True
            continue
        row = key[t]
        if groups > 1:
            m = E // groups
            total = []
            for g in range(groups):
                best = np.sort(row[g * m:(g + 1) * m])[::-1][:2]
                best = best[best > -np.inf].astype(np.float32)
                total.append(-np.inf if best.size == 0 else float(best.sum(dtype=np.float32)))
            order = sorted(range(groups), key=lambda g: (-total[g], g))[top_groups:]
            for g in order:
                row[g * m:(g + 1) * m] = -np.inf
        order = sorted(range(E), key=lambda e: (-row[e], e))[:k]
        for j, e in enumerate(order):
            if row[e] > -np.inf:
                ids[t, j] = e
    return ids, flagged


def shares(z, scoring):
    """Scores scaled to a sum of one; 0 for a row of -infinity."""
    z = np.asarray(z, np.float64)
    if scoring == "softmax":
        m = z.max(axis=1, keepdims=True)
        p = np.exp(z - np.where(np.isfinite(m), m, 0.0))
    else:
        # times e^-m, which leaves the ratios: nothing underflows
        m = np.minimum(z.max(axis=1, keepdims=True), 0.0)
        m = np.where(np.isfinite(m), m, 0.0)
        with np.errstate(over="ignore"):
            p = np.where(z >= 0, sigmoid(z) * np.exp(-m), np.exp(np.minimum(z, 0) - m) /
                         (1.0 + np.exp(np.minimum(z, 0))))
    s = p.sum(axis=1, keepdims=True)
    return p / np.where(s > 0, s, 1.0)


def weights(z, ids, scoring, renorm, scale):
    T, k = ids.shape
    out = np.zeros((T, k))
    for t in range(T):
        on = ids[t] >= 0
        if not on.any():
            continue
        zc = np.asarray(z[t, ids[t][on]], np.float64)[None]
        if renorm:
            w = shares(zc, scoring)[0]
        elif scoring == "softmax":
            w = shares(z[t:t + 1], scoring)[0][ids[t][on]]
        else:
            w = sigmoid(zc)[0]
        out[t, on] = w * np.float64(np.float32(scale))
    return out


def sequences(T, offsets):
    """Each token's sequence, -1 outside all."""
    seq = np.full(T, -1, np.int64)
    for s in range(len(offsets) - 1):
        seq[offsets[s]:offsets[s + 1]] = s
    return seq


def balance(z, ids, scoring, offsets):
    """loss [S], counts [S, E], tokens [S], mean [S, E]."""
    T, E = z.shape
    k, S = ids.shape[1], len(offsets) - 1
    p = shares(z, scoring)
    loss, mean = np.zeros(S), np.zeros((S, E))
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    for s in range(S):
        at = np.arange(offsets[s], offsets[s + 1])
        at = at[((ids[at] >= 0) & (ids[at] < E)).any(axis=1)]
        tokens[s] = len(at)
        if len(at) == 0:
            continue
        good = ids[at][(ids[at] >= 0) & (ids[at] < E)]
        counts[s] = np.bincount(good, minlength=E)
        mean[s] = p[at].sum(axis=0) / len(at)
        loss[s] = E / (k * len(at)) * (counts[s] * mean[s]).sum()
    return loss, counts, tokens, mean


def gradient(z, ids, scoring, renorm, scale, d_weights=None, d_loss=None, offsets=None):
    """(dz, size): the gradient and the sum of the absolute terms of each
    element, for the tolerance (for the balance loss after k T' / E is taken
    off the counts, which leaves the gradient as it is)."""
    T, E = z.shape
    k = ids.shape[1]
    z = np.asarray(z, np.float64)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    inner = np.ones((T, E)) if scoring == "softmax" else sigmoid(-z)
    p = shares(z, scoring)
    scale = np.float64(np.float32(scale))
    ok = (ids >= 0) & (ids < E)
    u = np.zeros((T, E))
    if d_weights is not None:
        for t in range(T):
            e = ids[t][ok[t]]
            if e.size == 0:
                continue
            g = np.asarray(d_weights[t][ok[t]], np.float64) * scale
            if renorm:
                q = shares(z[t, e][None], scoring)[0]
                np.add.at(d[t], e, inner[t, e] * q * (g - (q * g).sum()))
                np.add.at(size[t], e, inner[t, e] * q * (abs(g) + (q * abs(g)).sum()))
            elif scoring == "sigmoid":
                np.add.at(d[t], e, inner[t, e] * sigmoid(z[t, e]) * g)
                np.add.at(size[t], e, inner[t, e] * sigmoid(z[t, e]) * abs(g))
            else:
                np.add.at(u[t], e, g)
    if d_loss is not None:
        seq = sequences(T, offsets)
        _, counts, tokens, _ = balance(z, ids, scoring, offsets)
        for t in range(T):
            s = seq[t]
            if s >= 0 and ok[t].any():
                n = tokens[s]
                u[t] += float(d_loss[s]) * E / (k * n * n) * (counts[s] - k * n / E)
    dot = (p * u).sum(axis=1, keepdims=True)
    live = ok.any(axis=1, keepdims=True)
    d += live * inner * p * (u - dot)
    size += live * inner * p * (abs(u) + (p * abs(u)).sum(axis=1, keepdims=True))
    return d, size


def weight_values(fmt, codes, scales):
    """[..., H / 2] codes and [..., groups] scale bytes -> [..., H] values."""
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], axis=-1)
    v = v.reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    b = scales.astype(np.int64)
    if fmt == "mxfp4":
        s = np.where(b == 255, np.nan, 2.0 ** (b - 127.0))
    else:
        mag, sign = b & 127, np.where(b >= 128, -1.0, 1.0)
        top, low = mag >> 3, mag & 7
        s = np.where(top > 0, (8 + low) * 2.0 ** (top - 10.0), low * 2.0 ** -9) * sign
        s = np.where(mag == 127, np.nan, s)
    blk = v.shape[-1] // s.shape[-1]
    return v * np.repeat(s, blk, axis=-1)
