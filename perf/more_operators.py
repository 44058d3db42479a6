"""The operators of a dense layer and of a head that scores tokens, as measured cases.

Each case is one pass through one operator: the product of activations with block-scaled weights that leaves with bias,
activation, dropout and residual applied; the backward pass of that epilogue; dropout by itself; the log probabilities
of given tokens with entropy and alternatives; and their gradient.  With ``own`` false a pass is computed in plain torch
operations in 32 bits; with ``own`` true it is the calls of this repository's package.  ``exact`` gives the same results
from the definitions in 64 bits.

Sizes follow the repository's workloads (hidden sizes 4096 and 7168, inner sizes 2048 and 14336, batches of 4096 and
16384 tokens), with smaller, odd and single-token ones around them; vocabularies are generic.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WEIGHTS = ["mxfp4", "nvfp4", "mxfp8", "mxfp8_e5m2", "mxint8"]
ACTIVATIONS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# --- cases -----------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step, back from the inner size to the residual stream: latency and the weights' bytes
        {"name": "linear_one_token", "op": "linear", "rows": 1, "n": 7168, "k": 2048, "weights": "nvfp4",
         "type": "bf16", "bias": "bf16", "act": "none", "keep_z": False, "drop": 0.0, "residual": True},
        # the tokens of a few requests decoded together, into the wide inner size
        {"name": "linear_few_tokens", "op": "linear", "rows": 37, "n": 14336, "k": 4096, "weights": "mxfp8",
         "type": "bf16", "bias": "bf16", "act": "silu", "keep_z": False, "drop": 0.0, "residual": False},
        # a training batch, back to the residual stream with dropout
        {"name": "linear_residual", "op": "linear", "rows": 4096, "n": 7168, "k": 2048, "weights": "nvfp4",
         "type": "bf16", "bias": "f32", "act": "none", "keep_z": False, "drop": 0.1, "residual": True},
        # a long training batch into the inner size; what the backward pass needs is kept
        {"name": "linear_inner", "op": "linear", "rows": 16384, "n": 14336, "k": 4096, "weights": "mxfp4",
         "type": "bf16", "bias": "f32", "act": "gelu", "keep_z": True, "drop": 0.0, "residual": False},
        # its backward pass: gradients of the product and of the bias
        {"name": "epilogue_backward_inner", "op": "epilogue_backward", "rows": 16384, "cols": 14336, "type": "bf16",
         "act": "gelu", "drop": 0.0},
        # the same with dropout in 32 bits, an odd number of rows and columns
        {"name": "epilogue_backward_odd", "op": "epilogue_backward", "rows": 4099, "cols": 2047, "type": "f32",
         "act": "silu", "drop": 0.1},
        # a handful of tokens: nothing but latency
        {"name": "dropout_few_tokens", "op": "dropout", "rows": 8, "cols": 4096, "type": "bf16", "drop": 0.1,
         "residual": False},
        # a training batch into the residual stream
        {"name": "dropout_residual", "op": "dropout", "rows": 16384, "cols": 7168, "type": "bf16", "drop": 0.1,
         "residual": True},
        # one token of a serving step with 20 alternatives, part of an odd vocabulary not allowed
        {"name": "logprob_one_token", "op": "logprob", "tokens": 1, "vocab": 50257, "type": "bf16", "topk": 20,
         "scale": 1.25, "masked": 0.1, "padding": 0.0},
        # a batch of answers scored, with a few alternatives each
        {"name": "logprob_batch", "op": "logprob", "tokens": 4096, "vocab": 128000, "type": "bf16", "topk": 5,
         "scale": 1.0, "masked": 0.0, "padding": 0.0},
        # the gradient of a policy loss with an entropy term over such a batch, part of it prompt and padding
        {"name": "logprob_backward_batch", "op": "logprob_backward", "tokens": 4096, "vocab": 128000, "type": "bf16",
         "scale": 1.0, "masked": 0.0, "padding": 0.1},
        # 32-bit scores of a shorter batch over an odd vocabulary, at a temperature
        {"name": "logprob_backward_odd", "op": "logprob_backward", "tokens": 509, "vocab": 50257, "type": "f32",
         "scale": 1.25, "masked": 0.1, "padding": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "epilogue_backward", "dropout", "logprob", "logprob",
                     "logprob_backward"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    drop = rng.choice([0.0, 0.1, 0.5])
    if op == "linear":
        n, k = _log(rng, 64, 14336), 32 * _log(rng, 4, 448)
        if rng.random() < 0.5:
            n = -(-n // 128) * 128
        rows = _log(rng, 1, min(16384, 9 * 10 ** 11 // (n * k)))
        return {"op": op, "rows": rows, "n": n, "k": k, "weights": rng.choice(WEIGHTS), "type": kind,
                "bias": rng.choice(["bf16", "f32", "none"]), "act": rng.choice(ACTIVATIONS),
                "keep_z": rng.random() < 0.5, "drop": drop, "residual": rng.random() < 0.5}
    if op in ("epilogue_backward", "dropout"):
        cols = _log(rng, 16, 14336)
        most = 16384 * (14336 if op == "epilogue_backward" else 7168) // (2 if kind == "f32" else 1)
        case = {"op": op, "rows": _log(rng, 1, min(16384, most // cols)), "cols": cols, "type": kind}
        if op == "dropout":
            return dict(case, drop=drop or 0.25, residual=rng.random() < 0.5)
        return dict(case, act=rng.choice(ACTIVATIONS[1:]), drop=drop)
    vocab = _log(rng, 1000, 128000)
    case = {"op": op, "tokens": _log(rng, 1, min(8192, 4096 * 128000 // (2 if kind == "f32" else 1) // vocab)),
            "vocab": vocab, "type": kind, "scale": rng.choice([1.0, 1.25, 0.5]),
            "masked": rng.choice([0.0, 0.0, 0.1, 0.9])}
    if op == "logprob":
        topk = rng.choice([0, 1, 5, 20])
        return dict(case, topk=topk, padding=0.0 if topk else rng.choice([0.0, 0.1, 0.5]))
    return dict(case, padding=rng.choice([0.0, 0.1, 0.5]))


# --- inputs ----------------------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device=DEVICE, generator=g)


def _uniform(g, *shape):
    return torch.rand(*shape, device=DEVICE, generator=g)


def _matrix(rows, cols, kind, values=None):
    """[rows, cols] with a row pitch that keeps rows 16-byte aligned."""
    unit = 16 // TYPES[kind].itemsize
    m = torch.empty(rows, -(-cols // unit) * unit, dtype=TYPES[kind], device=DEVICE)[:, :cols]
    if values is not None:
        m.copy_(values)
    return m


def _activation(g, rows, cols):
    """Activations with a few large columns, as in the repository's workloads."""
    x = _normal(g, rows, cols)
    return x.mul_(1 + 9 * (_uniform(g, cols) < 0.01).float())


def _power(e):
    """2^e in 32 bits, exactly, for e in -126 .. 127 (and 0 for -127, the scale of a block of zeros)."""
    return ((e.int() + 127) << 23).view(torch.float32)


FOUR = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of E2M1 codes 0 .. 7
BETWEEN = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _four_bit_codes(y):
    """Nearest E2M1 codes of y, two to a byte, the even element in the low half."""
    code = torch.bucketize(y.abs(), torch.tensor(BETWEEN, device=DEVICE)).to(torch.uint8)
    code |= (y < 0).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _encode(w, weights):
    """(codes, scales, tensor scale or None) of w [rows, cols] in a block format."""
    rows, cols = w.shape
    if weights == "nvfp4":
        b = w.view(rows, cols // 16, 16)
        s = (w.abs().max() / 2688).clamp(min=1e-30)
        block = (b.abs().amax(2) / (6 * s)).clamp(max=448).to(torch.float8_e4m3fn)
        unit = block.float()[:, :, None] * s
        codes = _four_bit_codes(torch.where(unit > 0, b / unit.clamp(min=1e-30), 0.0).view(rows, cols))
        return codes, block.view(torch.uint8), s.view(1)
    b = w.view(rows, cols // 32, 32)
    largest = b.abs().amax(2, keepdim=True)
    top = {"mxfp4": 2, "mxfp8": 8, "mxfp8_e5m2": 15, "mxint8": 0}[weights]
    e = torch.where(largest > 0, torch.frexp(largest).exponent - 1 - top, -127).clamp(-127, 127)
    y = (b * _power(-e)).view(rows, cols)
    if weights == "mxfp4":
        codes = _four_bit_codes(y)
    elif weights == "mxint8":
        codes = torch.round(y * 64).clamp(-128, 127).to(torch.int8).view(torch.uint8)
    else:
        of, limit = (torch.float8_e4m3fn, 448) if weights == "mxfp8" else (torch.float8_e5m2, 57344)
        codes = y.clamp(-limit, limit).to(of).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8).view(rows, cols // 32), None


def _scores(g, case):
    """Scores of a head: a preference for few entries, part of them not allowed (minus infinity)."""
    t, v = case["tokens"], case["vocab"]
    x = _normal(g, t, v).mul_(2).add_(_normal(g, v) * 2)
    if case["masked"]:
        x.masked_fill_(_uniform(g, t, v) < case["masked"], -math.inf)
    return torch.empty(t, v, dtype=TYPES[case["type"]], device=DEVICE).copy_(x)


def _targets(g, logits, padding):
    """The tokens that were sampled: entries that are allowed; -1 for padding."""
    noisy = logits.float()
    noisy -= torch.log(-torch.log(_uniform(g, *logits.shape).clamp(1e-20, 1 - 1e-7)))
    target = noisy.argmax(1)
    return torch.where(_uniform(g, len(target)) < padding, -1, target)


def _stream_of(seed, op):
    """Seed and counter of the random stream."""
    return 0x9E3779B97F4A7C15 * (seed + 1) % 2 ** 63, 1000003 * seed + len(op)


def prepare(case, seed):
    g, op, kind = _generator(seed), case["op"], case["type"]
    s = {"case": case, "stream": _stream_of(seed, op)}
    if op == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        s["x"] = _matrix(m, k, "bf16", _activation(g, m, k))
        s["codes"], s["scales"], s["tensor_scale"] = _encode(_normal(g, n, k).mul_(0.02), case["weights"])
        s["bias"] = None if case["bias"] == "none" else _normal(g, n).to(TYPES[case["bias"]])
        s["residual"] = _matrix(m, n, kind, _normal(g, m, n)) if case["residual"] else None
        s["z"] = _matrix(m, n, kind) if case["keep_z"] else None
        s["out"] = _matrix(m, n, kind)
        if own:
            import microscaling_precision_gemm_amd as mx
            s["weights"] = mx.MXTensor(mx.FORMATS[case["weights"]], n, k, s["codes"], s["scales"], s["tensor_scale"])
    elif op == "epilogue_backward":
        m, n = case["rows"], case["cols"]
        s["z"], s["d_out"] = _matrix(m, n, kind, _normal(g, m, n)), _matrix(m, n, kind, _normal(g, m, n) * 0.01)
        s["d_z"], s["d_bias"] = _matrix(m, n, kind), torch.empty(n, device=DEVICE)
        if own:
            import microscaling_precision_gemm_amd as mx
            s["workspace"] = torch.empty(mx.mx_epilogue_workspace_bytes(m, n), dtype=torch.uint8, device=DEVICE)
    elif op == "dropout":
        m, n = case["rows"], case["cols"]
        s["x"] = _matrix(m, n, kind, _normal(g, m, n))
        s["residual"] = _matrix(m, n, kind, _normal(g, m, n)) if case["residual"] else None
        s["out"] = _matrix(m, n, kind)
    else:
        t, v = case["tokens"], case["vocab"]
        s["logits"] = _scores(g, case)
        s["target"] = _targets(g, s["logits"], case["padding"])
        if op == "logprob_backward":
            # what the forward pass left behind, and the gradients that arrive
            s["forward"] = _logprob(s["logits"], s["target"], case["scale"], 0)
            s["d_logp"], s["d_entropy"] = _normal(g, t) / t, torch.full((t,), -0.01 / t, device=DEVICE)
            s["d_logits"] = torch.empty_like(s["logits"])
        if own:
            import microscaling_precision_gemm_amd as mx
            s["buffers"] = mx.logprobs(t, v, case.get("topk", 0))
            if op == "logprob_backward":
                for name in ("entropy", "row_max", "log_sum"):
                    getattr(s["buffers"], name).copy_(s["forward"][name])
    return s


# --- plain forms -----------------------------------------------------------------------------------------------------
def _decode(s):
    """The weights' values in 32 bits."""
    c = s["case"]
    n, k, weights = c["n"], c["k"], c["weights"]
    if weights in ("mxfp4", "nvfp4"):
        table = torch.tensor(FOUR + tuple(-v for v in FOUR), device=DEVICE)
        v = torch.stack([table[(s["codes"] & 15).int()], table[(s["codes"] >> 4).int()]], dim=2)
    elif weights == "mxint8":
        v = s["codes"].view(torch.int8).float() / 64
    else:
        v = s["codes"].view(torch.float8_e4m3fn if weights == "mxfp8" else torch.float8_e5m2).float()
    if weights == "nvfp4":
        unit = s["scales"].view(torch.float8_e4m3fn).float()[:, :, None]
        return (v.view(n, k // 16, 16) * unit * s["tensor_scale"]).view(n, k)
    return (v.view(n, k // 32, 32) * _power(s["scales"].int()[:, :, None] - 127)).view(n, k)


def _keep(stream, rows, cols, drop):
    """(which elements stay, what they are multiplied by): 16 bits of Philox-4x32-10 an element."""
    seed, counter = stream
    groups = -(-cols // 8)
    at = torch.arange(rows * groups, dtype=torch.int64, device=DEVICE) + counter
    low = 0xFFFFFFFF
    c0, c1, c2, c3 = at & low, at >> 32 & low, torch.zeros_like(at), torch.zeros_like(at)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits, as the halves below need them
        c0, c1, c2, c3 = (p1 >> 32 & low) ^ c1 ^ k0, p1 & low, (p0 >> 32 & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([half for word in (c0, c1, c2, c3) for half in (word & 0xFFFF, word >> 16)], dim=1)
    threshold = round(drop * 65536)
    return bits.view(rows, groups * 8)[:, :cols] >= threshold, 65536 / (65536 - threshold)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":  # 0.5 z (1 + tanh u)
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-u * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * u * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _linear(s):
    c = s["case"]
    z = s["x"].float() @ _decode(s).t()
    if s["bias"] is not None:
        z += s["bias"].float()
    out = {"z": z.to(TYPES[c["type"]])} if c["keep_z"] else {}
    y = _act(z, c["act"])
    if c["drop"]:
        keep, factor = _keep(s["stream"], c["rows"], c["n"], c["drop"])
        y = torch.where(keep, y * factor, 0.0)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return dict(out, out=y.to(TYPES[c["type"]]))


def _logprob(logits, target, scale, topk):
    x = logits.float()
    m = x.amax(1)
    d = ((x - m[:, None]) * scale).clamp(min=-150)
    e = torch.exp(d)
    total = e.sum(1)
    log_sum = torch.log(total)
    there = target >= 0
    at = target.clamp(min=0)[:, None]
    logp = (torch.gather(x, 1, at)[:, 0] - m) * scale - log_sum
    out = {"logp": torch.where(there, logp, 0.0), "row_max": torch.where(there, m, 0.0),
           "entropy": torch.where(there, log_sum - (e * d).sum(1) / total, 0.0),
           "log_sum": torch.where(there, log_sum, 0.0)}
    if topk:
        ids, left = [], x.clone()
        for _ in range(topk):
            ids.append(left.argmax(1))  # ties: the lowest index
            left.scatter_(1, ids[-1][:, None], -math.inf)
        ids = torch.stack(ids, dim=1)
        out["top_id"] = ids.int()
        out["top_logp"] = (torch.gather(x, 1, ids) - m[:, None]) * scale - log_sum[:, None]
    return out


def _logprob_backward(s):
    c, f = s["case"], s["forward"]
    lp = (s["logits"].float() - f["row_max"][:, None]) * c["scale"] - f["log_sum"][:, None]
    p = torch.exp(lp)
    d = -s["d_logp"][:, None] * p - s["d_entropy"][:, None] * p * (lp.clamp(min=-150) + f["entropy"][:, None])
    d.scatter_add_(1, s["target"].clamp(min=0)[:, None], s["d_logp"][:, None])
    d = torch.where(s["target"][:, None] >= 0, d * c["scale"], 0.0)
    return {"d_logits": d.to(s["logits"].dtype)}


def _plain(s):
    c = s["case"]
    op, kind = c["op"], c["type"]
    if op == "linear":
        return _linear(s)
    if op == "logprob":
        return _logprob(s["logits"], s["target"], c["scale"], c["topk"])
    if op == "logprob_backward":
        return _logprob_backward(s)
    if op == "epilogue_backward":
        d = s["d_out"].float() * _act_slope(s["z"].float(), c["act"])
        if c["drop"]:
            keep, factor = _keep(s["stream"], c["rows"], c["cols"], c["drop"])
            d = torch.where(keep, d * factor, 0.0)
        return {"d_z": d.to(TYPES[kind]), "d_bias": d.sum(0)}
    keep, factor = _keep(s["stream"], c["rows"], c["cols"], c["drop"])
    y = torch.where(keep, s["x"].float() * factor, 0.0)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return {"out": y.to(TYPES[kind])}


# --- the library's calls ---------------------------------------------------------------------------------------------
def _own(s):
    import microscaling_precision_gemm_amd as mx
    c, (seed, counter) = s["case"], s["stream"]
    op = c["op"]
    if op in ("linear", "epilogue_backward"):
        act = mx.ACTIVATIONS[c["act"]]
    if op == "linear":
        mx.mx_linear(s["x"], s["weights"], s["out"], bias=s["bias"], act=act, z=s["z"], residual=s["residual"],
                     drop=c["drop"], seed=seed, counter=counter)
        return {"z": s["z"], "out": s["out"]} if c["keep_z"] else {"out": s["out"]}
    if op == "epilogue_backward":
        mx.mx_epilogue_backward(s["d_out"], s["z"], s["d_z"], s["d_bias"], act=act, drop=c["drop"], seed=seed,
                                counter=counter, workspace=s["workspace"])
        return {"d_z": s["d_z"], "d_bias": s["d_bias"]}
    if op == "dropout":
        return {"out": mx.mx_dropout(s["x"], s["out"], c["drop"], seed=seed, counter=counter, residual=s["residual"])}
    if op == "logprob":
        b = mx.mx_logprob(s["logits"], s["target"], s["buffers"], scale=c["scale"])
        out = {"logp": b.logp, "row_max": b.row_max, "entropy": b.entropy, "log_sum": b.log_sum}
        return dict(out, top_id=b.top_id, top_logp=b.top_logp) if c["topk"] else out
    return {"d_logits": mx.mx_logprob_backward(s["logits"], s["target"], s["buffers"], s["d_logp"], s["d_entropy"],
                                               s["d_logits"], scale=c["scale"])}


def run(state):
    return _own(state) if own else _plain(state)


# --- what a pass cannot do without -----------------------------------------------------------------------------------
def work(case):
    op, size = case["op"], TYPES[case["type"]].itemsize
    if op == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        weight = n * k // 2 + n * k // (16 if case["weights"] == "nvfp4" else 32)
        if case["weights"] not in ("mxfp4", "nvfp4"):
            weight += n * k // 2
        bias = n * {"none": 0, "bf16": 2, "f32": 4}[case["bias"]]
        return {"bytes": 2 * m * k + weight + bias + size * m * n * (1 + case["keep_z"] + case["residual"]),
                "flops": 2 * m * n * k}
    if op == "epilogue_backward":
        return {"bytes": 3 * size * case["rows"] * case["cols"] + 4 * case["cols"],
                "flops": 10 * case["rows"] * case["cols"]}
    if op == "dropout":
        return {"bytes": (2 + case["residual"]) * size * case["rows"] * case["cols"],
                "flops": 2 * case["rows"] * case["cols"]}
    looked_at = round(case["tokens"] * (1 - case["padding"])) * case["vocab"]
    if op == "logprob":
        return {"bytes": size * looked_at + case["tokens"] * (24 + 8 * case["topk"]), "flops": 6 * looked_at}
    return {"bytes": size * (looked_at + case["tokens"] * case["vocab"]) + 28 * case["tokens"],
            "flops": 8 * looked_at}


# --- the definitions in 64 bits --------------------------------------------------------------------------------------
def _exact_weights(s):
    """The values that codes and scales stand for, from the bits."""
    c = s["case"]
    n, k, weights = c["n"], c["k"], c["weights"]
    two_to = lambda e: ((e.long() + 1023) << 52).view(torch.float64)

    def small_float(code, exponent, mantissa, bias):
        field, rest = code >> mantissa & (1 << exponent) - 1, (code & (1 << mantissa) - 1).double() / (1 << mantissa)
        v = torch.where(field == 0, 2 * rest, 1 + rest) * two_to(field - bias)
        return torch.where(code >> (exponent + mantissa) > 0, -v, v)

    codes = s["codes"].long()
    if weights in ("mxfp4", "nvfp4"):
        v = torch.empty(n, k, dtype=torch.float64, device=DEVICE)
        v[:, 0::2], v[:, 1::2] = small_float(codes & 15, 2, 1, 1), small_float(codes >> 4, 2, 1, 1)
    elif weights == "mxint8":
        v = torch.where(codes > 127, codes - 256, codes).double() / 64
    else:
        v = small_float(codes, 4, 3, 7) if weights == "mxfp8" else small_float(codes, 5, 2, 15)
    if weights == "nvfp4":
        unit = small_float(s["scales"].long(), 4, 3, 7) * s["tensor_scale"].double()
        return v * unit.repeat_interleave(16, dim=1)
    return v * two_to(s["scales"].long() - 127).repeat_interleave(32, dim=1)


def _exact_factors(stream, rows, cols, drop):
    """0 or 1 / (1 - p) for each element, p the probability in steps of 2^-16."""
    seed, counter = stream
    groups = (cols + 7) // 8
    word = [torch.arange(rows * groups, dtype=torch.int64, device=DEVICE) + counter]
    word = [word[0] % 2 ** 32, word[0] // 2 ** 32] + [torch.zeros_like(word[0])] * 2
    key = [seed % 2 ** 32, seed // 2 ** 32]

    def product(a, m):  # high and low word of a m, by halves of m
        top, bottom = a * (m // 65536), a * (m % 65536)
        total = top % 65536 * 65536 + bottom
        return top // 65536 + total // 2 ** 32, total % 2 ** 32

    for i in range(10):
        (h0, l0), (h1, l1) = product(word[0], 0xD2511F53), product(word[2], 0xCD9E8D57)
        word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    steps = round(drop * 65536)
    factor = torch.empty(rows * groups, 8, dtype=torch.float64, device=DEVICE)
    for j in range(8):
        draw16 = word[j // 2] // 65536 ** (j % 2) % 65536
        factor[:, j] = (draw16 >= steps).double() * (65536 / (65536 - steps))
    return factor.view(rows, groups * 8)[:, :cols]


def _exact_activation(z, act):
    """(value, slope)"""
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    if act in ("silu", "gelu_tanh"):
        a, b = (1.0, 0.0) if act == "silu" else (math.sqrt(8 / math.pi), 0.044715 * math.sqrt(8 / math.pi))
        s = torch.sigmoid(a * z + b * z ** 3)
        return z * s, s * (1 + z * torch.sigmoid(-(a * z + b * z ** 3)) * (a + 3 * b * z ** 2))
    if act == "gelu":
        normal = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * normal, normal + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op, kind = case["op"], case["type"]
    if op == "linear":
        z = s["x"].double() @ _exact_weights(s).t()
        if s["bias"] is not None:
            z += s["bias"].double()
        out, _ = _exact_activation(z, case["act"])
        if case["drop"]:
            out = out * _exact_factors(s["stream"], case["rows"], case["n"], case["drop"])
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return {"z": z, "out": out} if case["keep_z"] else {"out": out}
    if op == "epilogue_backward":
        d = _exact_activation(s["z"].double(), case["act"])[1] * s["d_out"].double()
        if case["drop"]:
            d *= _exact_factors(s["stream"], case["rows"], case["cols"], case["drop"])
        return {"d_z": d, "d_bias": d.sum(0)}
    if op == "dropout":
        out = s["x"].double() * _exact_factors(s["stream"], case["rows"], case["cols"], case["drop"])
        return {"out": out if s["residual"] is None else out + s["residual"].double()}
    t = case["tokens"]
    there = s["target"] >= 0
    parts = []
    for a in range(0, t, 512):  # (a part of the rows at a time)
        x, at = s["logits"][a:a + 512].double(), s["target"][a:a + 512]
        ok = there[a:a + 512]
        q = torch.log_softmax(x * case["scale"], dim=1)
        p = torch.exp(q)
        entropy = -torch.special.xlogy(p, p).sum(1)
        hot = torch.zeros_like(p).scatter_(1, at.clamp(min=0)[:, None], 1.0)
        if op == "logprob_backward":
            dl, dh = s["d_logp"][a:a + 512].double(), s["d_entropy"][a:a + 512].double()
            d = dl[:, None] * (hot - p) - dh[:, None] * (torch.special.xlogy(p, p) + p * entropy[:, None])
            parts.append({"d_logits": torch.where(ok[:, None], d * case["scale"], 0.0)})
            continue
        m = x.amax(1)
        lse = torch.logsumexp((x - m[:, None]) * case["scale"], dim=1)
        own_logp = torch.gather(q, 1, at.clamp(min=0)[:, None])[:, 0]
        part = {n: torch.where(ok, v, 0.0) for n, v in (("logp", own_logp), ("row_max", m), ("entropy", entropy),
                                                        ("log_sum", lse))}
        if case["topk"]:
            order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :case["topk"]]
            part["top_id"], part["top_logp"] = order.int(), torch.gather(q, 1, order)
        parts.append(part)
    return {n: torch.cat([part[n] for part in parts]) for n in parts[0]}
