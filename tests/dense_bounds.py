"""Bounds on the errors of the measured operators' results (perf/more_operators.py)
against its 64-bit definitions, on the device in 64 bits.

U = 2^-24 is half a step of FP32; results are rounded once more to their type.  The
activations' bounds are those that dense_ref.py derives."""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}
A, B = math.sqrt(8 / math.pi), 0.044715 * math.sqrt(8 / math.pi)
STEEPEST = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}
TINY = 2.0 ** -118  # activations and slopes below it may be 0


def act(z, kind):
    """(activation, bound of its FP32 error for an exact z)"""
    if kind == "relu":
        return z.clamp(min=0), torch.zeros_like(z)
    if kind == "silu":
        y = z * torch.sigmoid(z)
        return y, 8 * U * y.abs() + TINY
    if kind == "gelu":
        y = z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return y, 18 * U * y.abs() + TINY
    if kind == "gelu_tanh":
        u = A * z + B * z ** 3
        y = z * torch.sigmoid(u)
        return y, (8 + 4 * u.abs() * torch.sigmoid(-u)) * U * y.abs() + TINY
    return z, torch.zeros_like(z)


def act_slope_error(z, kind):
    if kind in ("none", "relu"):
        return torch.zeros_like(z)
    if kind == "silu":
        s, o = torch.sigmoid(z), torch.sigmoid(-z)
        return U * (12 * s + 20 * z.abs() * s * o) + TINY
    if kind == "gelu":
        p, d = 0.5 * torch.special.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return U * (20 * p + 12 * z.abs() * d) + TINY
    u = A * z + B * z ** 3
    s, o = torch.sigmoid(u), torch.sigmoid(-u)
    second = z.abs() * s * o * (A + 3 * B * z ** 2)
    return U * ((12 + 4 * u.abs() * o) * s + (24 + 8 * u.abs()) * second) + TINY


def stored(want, err, kind):
    h = HALF_STEP[kind]
    return err + h * (want.abs() + err)


def linear(case, x, w, bias, factors, residual):
    """{"z", "out"}: (value, bound) for x, w and the rest in 64 bits (None: none).  The
    sum is held to the library's 1e-5 sum |x w|."""
    kind = case["act"]
    z = x @ w.t()
    err = 1e-5 * (x.abs() @ w.abs().t()) + U * z.abs()  # (tensor scale)
    if bias is not None:
        z = z + bias
        err = err + U * z.abs()
    y, e = act(z, kind)
    e = e + STEEPEST[kind] * err
    if factors is not None:
        y = y * factors
        e = e * factors + 2 * U * y.abs()
    if residual is not None:
        y = y + residual
        e = e + U * (y.abs() + e)
    return {"z": (z, stored(z, err, case["type"])), "out": (y, stored(y, e, case["type"]))}


def epilogue_backward(case, d_out, z, factors, want):
    """Bounds of d_z and d_bias; a column's sum has at most as many roundings as rows."""
    d = want["d_z"]
    e = d_out.abs() * act_slope_error(z, case["act"])
    if factors is not None:
        e = e * factors
    e = e + 3 * U * d.abs()
    return {"d_z": stored(d, e, case["type"]), "d_bias": e.sum(0) + len(d) * U * (d.abs() + e).sum(0)}


def roundings(vocab):
    """Of a row's sums: 15 of 16 entries; each step of at most 256, run, lane (6), wave
    (8) and part (32) rescales, by a factor good to 2 U, and adds: 4 U."""
    steps = min(-(-vocab // 1024), 256)  # (a workgroup has 64 lanes at least)
    return 15 + 4 * (steps + vocab / 2 ** 20 + 6 + 8 + 32)


def scores(x, scale):
    """Of each row in 64 bits: d = scale (x - m), log S, its bound, entropy, its bound.
    d of FP32 operations is off by 3 U |d| (difference, factor, product), a term by that
    and the exponential's 2 U."""
    d = (x - x.amax(1, keepdim=True)) * scale
    log_sum = torch.logsumexp(d, 1)
    p = torch.exp(d - log_sum[:, None])
    seen = torch.where(p > 0, d, 0.0)
    mean, square = -(p * seen).sum(1), (p * seen * seen).sum(1)
    n = roundings(x.shape[1]) + 2
    a = U * (3 * mean + n) + 2 * U * log_sum
    entropy = log_sum + mean
    e = a + U * (3 * square + n * mean) + a * mean + 5 * U * entropy
    return d, log_sum, a, entropy, e


def log_probability(d, log_sum, a):
    """Bound of scale (x - m) - log S for entries with a probability."""
    return torch.where(d > -math.inf, a + U * (4 * d.abs() + 2 * (d - log_sum).abs()), 0.0)


def logprob_backward(case, x, target, d_logp, d_entropy, want):
    d, log_sum, a, entropy, e_entropy = (v if v.dim() == 2 else v[:, None] for v in scores(x, case["scale"]))
    lp = d - log_sum
    p = torch.exp(lp)
    safe = torch.where(p > 0, lp, 0.0)
    e_lp = a + U * (3 * torch.where(p > 0, d, 0.0).abs() + 2 * safe.abs())
    dl, dh = d_logp[:, None].abs(), d_entropy[:, None].abs()
    inner = dl + dh * (safe + entropy).abs()
    e = p * (inner * (e_lp + 8 * U) + dh * (e_lp + e_entropy))
    hot = torch.zeros_like(p).scatter_(1, target.clamp(min=0)[:, None], 1.0)
    # a p below 2^-126 may be 0: its whole term is lost
    e = case["scale"] * (e + 3 * U * dl * hot + torch.where(p < 2.0 ** -125, 2.0 ** -125 * inner, 0.0))
    e = torch.where((target >= 0)[:, None], e, 0.0)
    return e + HALF_STEP[case["type"]] * (want.abs() + e) + 2.0 ** -125
