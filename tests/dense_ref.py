"""Plain 64-bit definitions of the dense layer's operators and of token scoring,
with bounds on what FP32 arithmetic may add, for the tests (numpy; nothing here
calls the library)."""
import math

import numpy as np
from scipy.special import erfc, expit

U = 2.0 ** -24  # half a step of FP32
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}

FOUR = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def eight_bit_values(fmt):
    """The 256 values of an 8-bit element type (infinities and NaN as NaN)."""
    c = np.arange(256)
    if fmt == "mxint8":
        return np.where(c > 127, c - 256, c) / 64.0
    man, bias = (3, 7) if fmt == "mxfp8" else (2, 15)
    e, m = (c & 127) >> man, (c & (1 << man) - 1) / (1 << man)
    v = np.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * 2.0 ** (e - bias))
    bad = (c & 127) == 127 if fmt == "mxfp8" else e == 31
    return np.where(bad, np.nan, np.where(c > 127, -v, v))


def weights(fmt, codes, scales, tensor_scale=1.0):
    """Values of the row layout's codes and scales."""
    if fmt in ("mxfp4", "nvfp4"):
        v = np.stack([FOUR[codes & 15], FOUR[codes >> 4]], axis=2).reshape(len(codes), -1)
    else:
        v = eight_bit_values(fmt)[codes]
    if fmt == "nvfp4":
        return v * np.repeat(eight_bit_values("mxfp8")[scales], 16, axis=1) * float(tensor_scale)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def draws(seed, counter, rows, cols):
    """16 bits for each element of a [rows, cols] matrix."""
    m32 = np.uint64(0xFFFFFFFF)
    groups = -(-cols // 8)
    at = np.uint64(counter) + np.arange(rows * groups, dtype=np.uint64)
    c = [at & m32, at >> np.uint64(32), np.zeros_like(at), np.zeros_like(at)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m32, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             p0 & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=1)
    return bits.reshape(rows, groups * 8)[:, :cols]


def drop_factors(drop, seed, counter, rows, cols):
    """What each element is multiplied by: 0 or 65536 / (65536 - t)."""
    t = min(int(np.rint(drop * 65536)), 65535)
    return np.where(draws(seed, counter, rows, cols) < t, 0.0, 65536.0 / (65536 - t))


# --- activations -------------------------------------------------------------
A, B = math.sqrt(8 / math.pi), 0.044715 * math.sqrt(8 / math.pi)


def act(z, kind):
    """(value, bound of the FP32 error for an exact z)

    silu: the sigmoid 5 U, the product U.  gelu: the tail's polynomial 9 U, the
    exponential 3 U, the square's correction 2 U, three products 3 U; above 0 one
    minus it, U more.  gelu_tanh: u takes 4 roundings, worth 4 |u| (1 - s) U of the
    sigmoid, then as silu.  Results below 2^-118 may be 0."""
    if kind == "relu":
        return np.maximum(z, 0), 0 * z
    if kind == "silu":
        y = z * expit(z)
        return y, 8 * U * np.abs(y) + 2.0 ** -118
    if kind == "gelu":
        y = z * 0.5 * erfc(-z / math.sqrt(2))
        return y, 18 * U * np.abs(y) + 2.0 ** -118
    if kind == "gelu_tanh":
        u = A * z + B * z ** 3
        y = z * expit(u)
        return y, (8 + 4 * np.abs(u) * expit(-u)) * U * np.abs(y) + 2.0 ** -118
    return z, 0 * z


def act_slope(z, kind):
    """(slope, bound of the FP32 error): the terms of the sum with the relative
    errors of their factors (7 U for s and 1 - s, as above for the others)."""
    if kind == "relu":
        return (z > 0).astype(float), 0 * z
    if kind == "silu":
        s, o = expit(z), expit(-z)
        return s + z * s * o, U * (12 * s + 20 * np.abs(z) * s * o) + 2.0 ** -118
    if kind == "gelu":
        p, d = 0.5 * erfc(-z / math.sqrt(2)), np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return p + z * d, U * (20 * p + 12 * np.abs(z) * d) + 2.0 ** -118
    if kind == "gelu_tanh":
        u, slope = A * z + B * z ** 3, A + 3 * B * z ** 2
        s, o = expit(u), expit(-u)
        second = np.abs(z) * s * o * slope
        return s + z * s * o * slope, U * ((12 + 4 * np.abs(u) * o) * s + (24 + 8 * np.abs(u)) * second) + 2.0 ** -118
    return np.ones_like(z), 0 * z


STEEPEST = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}


def linear(x, w, bias, kind, factors, residual, dtype):
    """((z, bound), (out, bound)) of the stored values.  The sum is held to the
    library's 1e-5 sum |x w|."""
    z = x @ w.T
    err = 1e-5 * (np.abs(x) @ np.abs(w).T) + U * np.abs(z)  # (tensor scale)
    if bias is not None:
        z = z + bias
        err = err + U * np.abs(z)
    y, e = act(z, kind)
    e = e + STEEPEST[kind] * err
    if factors is not None:
        y = y * factors
        e = e * factors + 2 * U * np.abs(y)
    if residual is not None:
        y = y + residual
        e = e + U * (np.abs(y) + e)
    h = HALF_STEP[dtype]
    return (z, err + h * (np.abs(z) + err)), (y, e + h * (np.abs(y) + e))


def epilogue_backward(d_out, z, kind, factors, dtype):
    """((d_z, bound), (d_bias, bound)); a column's sum has at most as many
    roundings as rows, and each term its own error."""
    s, e = act_slope(z, kind)
    d = d_out * s
    e = np.abs(d_out) * e + U * np.abs(d)
    if factors is not None:
        d = d * factors
        e = e * factors + 2 * U * np.abs(d)
    h = HALF_STEP[dtype]
    return (d, e + h * (np.abs(d) + e)), (d.sum(0), e.sum(0) + len(d) * U * (np.abs(d) + e).sum(0))


# --- token scoring -----------------------------------------------------------
def logprob(x, target, scale, topk, steps=64):
    """Results of each row and bounds of the FP32 ones.

    d = s (x - m) has a relative error of 3 U (difference, scale, product), so a
    term e^d one of (3 |d| + 3) U; a lane's running sum adds and rescales at most
    `steps` times, 12 U each, the joins of lanes and waves 22 more.  With E the mean
    under p: log S is off by a = (3 E|d| + 3 + 12 steps + 12 * 22) U and its own
    rounding; the mean of d by (3 E d^2 + ...) U likewise."""
    T, V = x.shape
    out = {k: np.zeros(T) for k in ("logp", "entropy", "row_max", "log_sum")}
    tol = {k: np.zeros(T) for k in out}
    ids, lps, lpt = np.full((T, topk), -1), np.full((T, topk), -np.inf), np.zeros((T, topk))
    n = 3 + 12 * (steps + 22)
    for t in range(T):
        row = x[t]
        if target is not None and not 0 <= target[t] < V:
            continue
        order = [v for v in np.argsort(-np.where(np.isnan(row), -np.inf, row), kind="stable")[:topk + 1]
                 if row[v] > -np.inf][:topk]
        ids[t, :len(order)] = order
        if np.isnan(row).any() or (row == np.inf).any():
            for k in out:
                out[k][t] = np.nan
            lps[t, :len(order)] = np.nan
            continue
        m = row.max()
        out["row_max"][t] = m
        if m == -np.inf:
            out["logp"][t] = -np.inf
            continue
        d = scale * (row - m)
        e = np.exp(d)
        S = e.sum()
        dd = np.where(e > 0, d, 0.0)
        mean, square = (e * -dd).sum() / S, (e * dd * dd).sum() / S
        ls = math.log(S)
        a = U * (3 * mean + n) + 2 * U * ls
        out["log_sum"][t], tol["log_sum"][t] = ls, a
        out["entropy"][t] = ls + mean
        tol["entropy"][t] = a + U * (3 * square + n * mean) + a * mean + 5 * U * (ls + mean)
        lp = lambda v: (d[v] - ls, a + 4 * U * abs(d[v]) + 2 * U * abs(d[v] - ls)) if row[v] > -np.inf else (-np.inf, 0)
        if target is not None:
            out["logp"][t], tol["logp"][t] = lp(target[t])
        for j, v in enumerate(order):
            lps[t, j], lpt[t, j] = lp(v)
    out.update(top_id=ids, top_logp=lps)
    tol["top_logp"] = lpt
    return out, tol


def logprob_backward(x, target, scale, d_logp, d_entropy, tol, dtype):
    """(d_x, bound); tol: the bounds of the saved statistics."""
    T, V = x.shape
    out, err = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        row = x[t]
        if target is not None and not 0 <= target[t] < V or (row == -np.inf).all():
            continue
        if np.isnan(row).any() or (row == np.inf).any():
            out[t] = np.nan
            continue
        d = scale * (row - row.max())
        ls = math.log(np.exp(d).sum())
        lp = d - ls
        p = np.exp(lp)
        safe = np.where(p > 0, lp, 0.0)
        H = -(p * safe).sum()
        dl = d_logp[t] if d_logp is not None and target is not None else 0.0
        dh = d_entropy[t] if d_entropy is not None else 0.0
        hot = np.zeros(V)
        if target is not None:
            hot[target[t]] = 1
        out[t] = scale * (dl * (hot - p) - dh * p * (safe + H))
        e_lp = tol["log_sum"][t] + U * (3 * np.abs(np.where(p > 0, d, 0.0)) + 2 * np.abs(safe))
        rel = e_lp + 4 * U  # of p
        inner = abs(dl) + abs(dh) * np.abs(safe + H)
        e = p * (inner * (rel + 4 * U) + abs(dh) * (e_lp + tol["entropy"][t]))
        # a p below 2^-126 may be 0: its whole term, p times at most `inner`, is lost
        e += 3 * U * abs(dl) * hot + np.where(p < 2.0 ** -125, 2.0 ** -125 * inner, 0.0)
        err[t] = scale * e
    err += HALF_STEP[dtype] * (np.abs(out) + err) + 2.0 ** -125
    return out, err
