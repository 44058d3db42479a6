"""The operators around the expert products of a mixture-of-experts layer, as measured cases.

Each case is one pass through one operator: the router with its dispatch order and balance loss, the gated activation
with its 8-bit checkpoint, the weight gradient that reads such a checkpoint, and the weighted combination of the
experts' rows.  With ``own`` false a pass is computed in plain torch operations in 32 bits; with ``own`` true it is the
calls of this repository's package.  ``exact`` gives the same results from the definitions in 64 bits.

Sizes follow the repository's mixture-of-experts workload (4096 tokens, hidden size 7168, 32 experts of inner size
2048, 8 experts a token) and its backward workload (16384 tokens), with smaller, odd and single-token ones around them.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --- cases -----------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step: nothing but latency
        {"name": "route_one_token", "op": "route", "tokens": 1, "experts": 32, "topk": 8, "type": "bf16",
         "normalize": True, "padding": 0.0},
        # the layer's training batch, scores kept in 32 bits as routers usually do
        {"name": "route_layer", "op": "route", "tokens": 4096, "experts": 32, "topk": 8, "type": "f32",
         "normalize": False, "padding": 0.0},
        # a long batch over many experts, with padding tokens that go nowhere
        {"name": "route_many_experts", "op": "route", "tokens": 16384, "experts": 256, "topk": 8, "type": "bf16",
         "normalize": True, "padding": 0.1},
        # the router's backward pass: gradients of the combine weights and of the balance loss
        {"name": "route_backward", "op": "route_backward", "tokens": 16384, "experts": 256, "topk": 8, "type": "f32",
         "normalize": True, "padding": 0.1},
        # the activation between the two expert products for one token's 8 experts
        {"name": "swiglu_one_token", "op": "swiglu", "rows": 8, "cols": 2048, "type": "bf16"},
        # the layer's training step of it: forward saving 8 bits, backward from them
        {"name": "swiglu_step", "op": "swiglu_step", "rows": 32768, "cols": 2048, "type": "bf16", "saved": "mxfp8"},
        # the same over an odd number of rows, 32-bit values, 8-bit integers saved
        {"name": "swiglu_step_odd", "op": "swiglu_step", "rows": 4099, "cols": 4096, "type": "f32", "saved": "mxint8"},
        # a few ragged experts, some without a row
        {"name": "wgrad_small", "op": "wgrad", "rows": 1003, "groups": 8, "n": 520, "k": 1024, "gather": False,
         "type": "bf16", "saved": "mxfp8"},
        # the layer's first weight gradient: saved tokens gathered by the dispatch order, 32-bit gradients
        {"name": "wgrad_layer", "op": "wgrad", "rows": 32768, "groups": 32, "n": 2048, "k": 7168, "gather": True,
         "type": "f32", "saved": "mxfp8"},
        # one token's 8 expert rows
        {"name": "combine_one_token", "op": "combine", "tokens": 1, "topk": 8, "cols": 7168, "type": "bf16"},
        # the layer's batch
        {"name": "combine_layer", "op": "combine", "tokens": 4096, "topk": 8, "cols": 7168, "type": "bf16"},
        # its backward pass, an odd number of tokens
        {"name": "combine_backward", "op": "combine_backward", "tokens": 4001, "topk": 8, "cols": 7168,
         "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "swiglu", "swiglu_step", "wgrad", "wgrad", "combine",
                     "combine_backward"])
    kind = rng.choice(["bf16", "f32"])
    if op in ("route", "route_backward"):
        experts = _log(rng, 4, 256)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "type": kind, "normalize": rng.random() < 0.5, "padding": rng.choice([0.0, 0.1, 0.5])}
    if op in ("swiglu", "swiglu_step"):
        cols = 32 * _log(rng, 1, 128)
        case = {"op": op, "rows": _log(rng, 1, min(32768, (32768 * 2048 // (2 if kind == "f32" else 1)) // cols)),
                "cols": cols, "type": kind}
        return case if op == "swiglu" else dict(case, saved=rng.choice(["mxfp8", "mxint8"]))
    if op == "wgrad":
        rows, groups = _log(rng, 16, 32768), _log(rng, 1, 32)
        k, n = 32 * _log(rng, 2, 224), 8 * _log(rng, 4, 256)
        return {"op": op, "rows": rows, "groups": groups, "n": n, "k": k, "gather": rng.random() < 0.5, "type": kind,
                "saved": rng.choice(["mxfp8", "mxint8"])}
    tokens = _log(rng, 1, 4001)
    cols = _log(rng, 64, 7168)
    if kind == "f32":
        tokens = min(tokens, 2000)
    return {"op": op, "tokens": tokens, "topk": rng.randint(1, 8), "cols": cols, "type": kind}


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


def _logits(g, case):
    """Scores of a router in training: a preference for some experts, and noise per token."""
    t, e = case["tokens"], case["experts"]
    return _matrix(t, e, case["type"], _normal(g, t, e) + 0.5 * _normal(g, e))


def _token_mask(g, case):
    """1 for a token, 0 for padding; None where the batch has none."""
    return (_uniform(g, case["tokens"]) >= case["padding"]).to(torch.uint8) if case["padding"] else None


def _activation(g, rows, cols):
    """Activations with a few large columns, as in the repository's workloads."""
    x = _normal(g, rows, cols)
    return x.mul_(1 + 9 * (_uniform(g, cols) < 0.01).float())


def _choices(g, tokens, experts, topk):
    """topk distinct experts for each token, some experts preferred."""
    return (_normal(g, tokens, experts) + 0.5 * _normal(g, experts)).topk(topk, dim=1).indices


def _dispatch(choice, experts):
    """(row_index, group_offsets, slot_row) of routed rows sorted by expert, tokens in order within one."""
    tokens, topk = choice.shape
    order = torch.argsort(choice.reshape(-1), stable=True)
    slot_row = torch.empty(tokens * topk, dtype=torch.int32, device=DEVICE)
    slot_row[order] = torch.arange(tokens * topk, dtype=torch.int32, device=DEVICE)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=DEVICE)
    offsets[1:] = torch.bincount(choice.reshape(-1), minlength=experts).cumsum(0)
    return (order // topk).to(torch.int32), offsets, slot_row.view(tokens, topk)


def prepare(case, seed):
    g, op, kind = _generator(seed), case["op"], case.get("type")
    s = {"case": case}
    if op in ("route", "route_backward"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s["logits"], s["mask"] = _logits(g, case), _token_mask(g, case)
        if op == "route_backward":
            # what the forward pass left behind, and the gradients that arrive
            f = _route(s["logits"], s["mask"], k, case["normalize"])
            s["forward"] = {n: f[n] for n in ("experts", "counts", "valid")}
            s["d_weights"] = _normal(g, t, k) * 0.01
            s["d_loss"] = torch.full((1,), 0.01, device=DEVICE)
            s["d_logits"] = _matrix(t, e, kind)
    elif op in ("swiglu", "swiglu_step"):
        r, c = case["rows"], case["cols"]
        s["h"] = _matrix(r, 2 * c, kind, _activation(g, r, 2 * c))
        s["y"], s["amax"] = _matrix(r, c, kind), torch.zeros(1, device=DEVICE)
        if op == "swiglu_step":
            s["codes"] = torch.empty(r, 2 * c, dtype=torch.uint8, device=DEVICE)
            s["scales"] = torch.empty(r, c // 16, dtype=torch.uint8, device=DEVICE)
            s["dy"], s["dh"] = _matrix(r, c, kind, _normal(g, r, c) * 0.01), _matrix(r, 2 * c, kind)
    elif op == "wgrad":
        r, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        topk = min(8, groups) if case["gather"] else 1
        tokens = -(-r // topk)
        choice = _choices(g, tokens, groups, topk)
        s["row_index"], s["offsets"], _ = _dispatch(choice, groups)
        r = s["rows"] = tokens * topk
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        if not case["gather"]:
            s["row_index"] = None
        s["codes"], s["scales"] = _encode(_activation(g, tokens, k), case["saved"])
        s["dy"] = _matrix(r, n, "bf16", _normal(g, r, n) * 0.01)
        s["dw"] = torch.empty(groups * n, k, dtype=TYPES[kind], device=DEVICE)
    else:
        t, k, c = case["tokens"], case["topk"], case["cols"]
        choice = _choices(g, t, 32, k)
        _, _, s["slot_row"] = _dispatch(choice, 32)
        s["rows"] = _matrix(t * k, c, kind, _normal(g, t * k, c))
        w = _uniform(g, t, k) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        if op == "combine":
            s["out"] = _matrix(t, c, kind)
        else:
            s["d_out"] = _matrix(t, c, kind, _normal(g, t, c) * 0.01)
            s["d_rows"], s["d_weights"] = _matrix(t * k, c, kind), torch.empty(t, k, device=DEVICE)
    return s


# --- plain forms -----------------------------------------------------------------------------------------------------
def _softmax(logits, mask):
    """Probabilities of each row; padding rows, and entries at minus infinity, have none."""
    x = logits.float()
    if mask is not None:
        x = torch.where(mask.bool()[:, None], x, -math.inf)
    m = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return x, p / p.sum(1, keepdim=True).clamp(min=1e-30)


def _route(logits, mask, topk, normalize):
    t, e = logits.shape
    x, p = _softmax(logits, mask)
    order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :topk]  # ties: the lower index first
    there = torch.gather(x, 1, order) > -math.inf
    w = torch.where(there, torch.gather(p, 1, order), 0.0)
    if normalize:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    chosen = torch.where(there, order, e)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    counts.index_add_(0, chosen.reshape(-1), torch.ones_like(chosen).reshape(-1))
    counts[e] = 0
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    offsets[1:] = counts[:e].cumsum(0)
    by_expert = torch.argsort(chosen.reshape(-1), stable=True)
    place = torch.empty_like(by_expert)
    place[by_expert] = torch.arange(t * topk, device=x.device)
    valid = torch.full((1,), t, dtype=torch.int64, device=x.device) if mask is None else mask.sum(dtype=torch.int64).view(1)
    prob_sum = p.sum(0)
    v = valid.float().clamp(min=1)
    loss = (counts[:e].float() * prob_sum).sum() * e / (topk * v * v)
    return {"experts": torch.where(there, order, -1).int(), "weights": w,
            "slot_row": torch.where(there, place.view(t, topk), -1).int(),
            "row_index": torch.where(chosen.reshape(-1)[by_expert] < e, by_expert // topk, -1).int(),
            "group_offsets": offsets, "counts": counts[:e], "valid": valid, "prob_sum": prob_sum, "loss": loss.view(1)}


def _route_backward(s):
    c, f = s["case"], s["forward"]
    e, k = c["experts"], c["topk"]
    _, p = _softmax(s["logits"], s["mask"])
    at = f["experts"].long().clamp(min=0)
    there = f["experts"] >= 0
    v = f["valid"].float().clamp(min=1)
    dp = (s["d_loss"] * e / (k * v * v) * f["counts"].float()).expand_as(p)
    dw = torch.where(there, s["d_weights"], 0.0)
    chosen = torch.where(there, torch.gather(p, 1, at), 0.0)
    if c["normalize"]:
        w = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
        dchosen = w * (dw - (w * dw).sum(1, keepdim=True))
    else:
        dchosen = None
        dp = dp.scatter_add(1, at, dw)
    dx = p * (dp - (p * dp).sum(1, keepdim=True))
    if dchosen is not None:
        dx = dx.scatter_add(1, at, torch.where(there, dchosen, 0.0))
    return dx.to(s["logits"].dtype)


def _power(e):
    """2^e in 32 bits, exactly, for e in -126 .. 127 (and 0 for -127, the scale of a block of zeros)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, saved):
    """(codes, scales) of x [rows, cols]: one power of two for 32 elements, 8-bit elements."""
    rows, cols = x.shape
    b = x.float().view(rows, cols // 32, 32)
    largest = b.abs().amax(2, keepdim=True)
    top = 8 if saved == "mxfp8" else 0
    e = torch.where(largest > 0, torch.frexp(largest).exponent - 1 - top, -127).clamp(-127, 127)
    y = b * _power(-e)
    if saved == "mxfp8":
        step = torch.frexp(y).exponent.clamp(min=-5) - 4  # three bits after the leading one, subnormals below 2^-6
        y = (torch.round(y * _power(-step)) * _power(step)).clamp(-448, 448)
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = torch.round(y * 64).clamp(-128, 127).to(torch.int8).view(torch.uint8)
    return codes.view(rows, cols), (e + 127).to(torch.uint8).view(rows, cols // 32)


def _decode(codes, scales, saved):
    rows, cols = codes.shape
    v = codes.view(torch.float8_e4m3fn).float() if saved == "mxfp8" else codes.view(torch.int8).float() / 64
    return (v.view(rows, cols // 32, 32) * _power(scales.int()[:, :, None] - 127)).view(rows, cols)


def _swiglu(h):
    gate, up = h.float().chunk(2, dim=1)
    return gate / (1 + torch.exp(-gate)) * up


def _swiglu_backward(h, dy):
    gate, up = h.chunk(2, dim=1)
    sig = 1 / (1 + torch.exp(-gate))
    dy = dy.float()
    return torch.cat([dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig], dim=1)


def _by_group(s, longest):
    """Row numbers [groups, longest] of each group's rows, and which of them are there."""
    lo, hi = s["offsets"][:-1, None], s["offsets"][1:, None]
    at = lo + torch.arange(longest, device=DEVICE)
    return at.clamp(max=max(s["rows"] - 1, 0)), at < hi


def _wgrad(s):
    c = s["case"]
    at, there = _by_group(s, s["longest"])
    src = at if s["row_index"] is None else s["row_index"].long()[at]
    x = _decode(s["codes"], s["scales"], c["saved"])[src]
    dy = torch.where(there[:, :, None], s["dy"].float()[at], 0.0)
    dw = torch.bmm(dy.transpose(1, 2).contiguous(), x)
    return dw.view(c["groups"] * c["n"], c["k"]).to(TYPES[c["type"]])


def _plain(s):
    c = s["case"]
    op, kind = c["op"], c.get("type")
    if op == "route":
        return _route(s["logits"], s["mask"], c["topk"], c["normalize"])
    if op == "route_backward":
        return {"d_logits": _route_backward(s)}
    if op in ("swiglu", "swiglu_step"):
        y = _swiglu(s["h"]).to(TYPES[kind])
        out = {"y": y, "amax": y.float().abs().amax().view(1)}
        if op == "swiglu_step":
            saved = _decode(*_encode(s["h"], c["saved"]), c["saved"])
            out["dh"] = _swiglu_backward(saved, s["dy"]).to(TYPES[kind])
        return out
    if op == "wgrad":
        return {"dw": _wgrad(s)}
    picked = s["rows"].float()[s["slot_row"].long()]
    if op == "combine":
        return {"out": (s["weights"][:, :, None] * picked).sum(1).to(TYPES[kind])}
    d_out = s["d_out"].float()[:, None, :]
    d_rows = torch.empty(s["rows"].shape, device=DEVICE)
    d_rows[s["slot_row"].reshape(-1).long()] = (s["weights"][:, :, None] * d_out).flatten(0, 1)
    return {"d_rows": d_rows.to(TYPES[kind]), "d_weights": (picked * d_out).sum(2)}


# --- the framework's operators ---------------------------------------------------------------------------------------
def _kernels(s):
    import microscaling_precision_gemm_amd as mx

    c = s["case"]
    op = c["op"]
    if op in ("route", "route_backward"):
        flags = mx.MX_ROUTE_NORMALIZE if c["normalize"] else 0
        r = s.get("routing")
        if r is None:  # the layer's buffers, kept from step to step
            r = s["routing"] = mx.routing(c["tokens"], c["experts"], c["topk"], device=DEVICE)
            for n, v in s.get("forward", {}).items():
                getattr(r, n).copy_(v)
        if op == "route":
            mx.mx_route(s["logits"], r, token_mask=s["mask"], flags=flags)
            return {n: getattr(r, n) for n in ("experts", "weights", "slot_row", "row_index", "group_offsets",
                                               "counts", "valid", "prob_sum", "loss")}
        mx.mx_route_backward(s["logits"], r, s["d_weights"], s["d_loss"], s["d_logits"], token_mask=s["mask"],
                             flags=flags)
        return {"d_logits": s["d_logits"]}
    if op == "swiglu":
        mx.mx_swiglu(s["h"], s["y"], amax=s["amax"])
        return {"y": s["y"], "amax": s["amax"]}
    if op == "swiglu_step":
        saved = mx.MXTensor(mx.FORMATS[c["saved"]], c["rows"], 2 * c["cols"], s["codes"], s["scales"])
        mx.mx_swiglu(s["h"], s["y"], saved=saved, amax=s["amax"])
        mx.mx_swiglu_backward(saved, s["dy"], s["dh"])
        return {"y": s["y"], "amax": s["amax"], "dh": s["dh"]}
    if op == "wgrad":
        x = mx.MXTensor(mx.FORMATS[c["saved"]], s["codes"].shape[0], c["k"], s["codes"], s["scales"])
        mx.mx_wgrad_grouped(s["dy"], x, s["row_index"], c["groups"], s["offsets"], s["dw"])
        return {"dw": s["dw"]}
    if op == "combine":
        mx.mx_combine(s["rows"], s["slot_row"], s["weights"], s["out"])
        return {"out": s["out"]}
    mx.mx_combine_backward(s["d_out"], s["rows"], s["slot_row"], s["weights"], s["d_rows"], s["d_weights"])
    return {"d_rows": s["d_rows"], "d_weights": s["d_weights"]}


def run(state):
    return _kernels(state) if own else _plain(state)


# --- what a pass cannot do without -----------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    b = TYPES[case["type"]].itemsize
    if op in ("route", "route_backward"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        mask = t if case["padding"] else 0
        if op == "route":
            return {"bytes": t * e * b + mask + 16 * t * k + 8 * (e + 1) + 12 * e + 12, "flops": 6 * t * e + 2 * t * k}
        return {"bytes": 2 * t * e * b + mask + 8 * t * k + 8 * e + 12, "flops": 9 * t * e + 4 * t * k}
    if op in ("swiglu", "swiglu_step"):
        n = case["rows"] * case["cols"]
        forward = {"bytes": 3 * n * b + 4, "flops": 6 * n}
        if op == "swiglu":
            return forward
        saved = 2 * n + n // 16  # codes and one scale for 32 of them, written once and read once
        return {"bytes": forward["bytes"] + 2 * saved + 3 * n * b, "flops": forward["flops"] + 10 * n + 12 * n}
    if op == "wgrad":
        r, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        topk = min(8, groups) if case["gather"] else 1
        tokens = -(-r // topk)
        r = tokens * topk
        return {"bytes": tokens * (k + k // 32) + r * n * 2 + groups * n * k * b + 4 * r * case["gather"]
                + 8 * (groups + 1), "flops": 2 * r * n * k}
    t, k, c = case["tokens"], case["topk"], case["cols"]
    if op == "combine":
        return {"bytes": t * k * (c * b + 8) + t * c * b, "flops": 2 * t * k * c}
    return {"bytes": 2 * t * k * c * b + 12 * t * k + t * c * b, "flops": 3 * t * k * c}


# --- the definitions in 64 bits --------------------------------------------------------------------------------------
def _exact_probabilities(logits, mask):
    x = logits.double()
    there = torch.isfinite(x)
    if mask is not None:
        there &= mask.bool()[:, None]
    p = torch.where(there, torch.exp(x - x.max(1, keepdim=True).values), 0.0)
    return there, p / p.sum(1, keepdim=True).clamp(min=1e-300)


def _exact_route(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["topk"]
    there, p = _exact_probabilities(s["logits"], s["mask"])
    # the order of the experts: larger score first, lower index first among equals
    rank = torch.sort(torch.where(there, -s["logits"].double(), math.inf), dim=1, stable=True).indices[:, :k]
    ok = there.gather(1, rank)
    w = p.gather(1, rank) * ok
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    picked = torch.zeros(t, e, dtype=torch.int64, device=DEVICE).scatter_add_(1, rank, ok.long())
    counts = picked.sum(0)
    start = counts.cumsum(0) - counts
    # a slot's row: its expert's start, and the earlier tokens of that expert
    slot = start[rank] + (picked.cumsum(0) - picked).gather(1, rank)
    row_index = torch.full((t * k,), -1, dtype=torch.int64, device=DEVICE)
    token = torch.arange(t, device=DEVICE)[:, None].expand(t, k)
    row_index[slot[ok]] = token[ok]
    valid = t if s["mask"] is None else int(s["mask"].sum())
    loss = e * (counts.double() / (k * max(valid, 1)) * (p.sum(0) / max(valid, 1))).sum()
    return {"experts": torch.where(ok, rank, -1), "weights": w, "slot_row": torch.where(ok, slot, -1),
            "row_index": row_index, "group_offsets": torch.cat([start, counts.sum().view(1)]), "counts": counts,
            "valid": torch.tensor([valid]), "prob_sum": p.sum(0), "loss": loss.view(1)}


def _exact_route_backward(s):
    c, f = s["case"], s["forward"]
    e, k = c["experts"], c["topk"]
    _, p = _exact_probabilities(s["logits"], s["mask"])
    valid = max(int(f["valid"]), 1)
    hot = torch.zeros(c["tokens"], e + 1, dtype=torch.float64, device=DEVICE)
    hot.scatter_(1, torch.where(f["experts"] < 0, e, f["experts"]).long(), s["d_weights"].double())
    is_hot = torch.zeros(c["tokens"], e + 1, device=DEVICE).scatter_(
        1, torch.where(f["experts"] < 0, e, f["experts"]).long(), 1.0)[:, :e].double()
    dw = hot[:, :e]
    balance = s["d_loss"].double() * e * f["counts"].double() / (k * valid * valid)
    d = p * (balance - (p * balance).sum(1, keepdim=True))
    if c["normalize"]:
        q = p * is_hot
        q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
        d += q * (dw - (q * dw).sum(1, keepdim=True))
    else:
        d += p * (dw - (p * dw).sum(1, keepdim=True))
    return d


def _two_to(e):
    """2^e in 64 bits, from the bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_saved(codes, scales, saved):
    """The values that 8-bit codes and their block scales stand for, from the bits."""
    c = codes.long()
    if saved == "mxint8":
        v = torch.where(c > 127, c - 256, c).double() / 64
    else:
        mag, field = (c & 7).double(), (c >> 3) & 15
        v = torch.where(field == 0, mag / 512, (1 + mag / 8) * _two_to(field - 7))
        v = torch.where(c > 127, -v, v)
    return v * _two_to(scales.long() - 127).repeat_interleave(32, dim=1)


def _exact_rounded(x, saved):
    """x as its 8-bit block format holds it: the block's largest power of two sets the grid."""
    rows, cols = x.shape
    b = x.double().view(rows, cols // 32, 32)
    largest = b.abs().amax(2, keepdim=True)
    unit = _two_to(torch.frexp(largest.clamp(min=2.0 ** -120)).exponent - 1 - (8 if saved == "mxfp8" else 0))
    q = b / unit
    if saved == "mxint8":
        q = (torch.round(q * 64) / 64).clamp(-2, 127 / 64)
    else:
        grid = _two_to(torch.frexp(q.abs().clamp(min=2.0 ** -6)).exponent - 4)
        q = (torch.round(q / grid) * grid).clamp(-448, 448)
    return (q * unit).view(rows, cols)


def exact(case, seed):
    s = prepare(case, seed)
    op, kind = case["op"], case["type"]
    if op == "route":
        return _exact_route(s)
    if op == "route_backward":
        return {"d_logits": _exact_route_backward(s)}
    if op in ("swiglu", "swiglu_step"):
        c = case["cols"]
        h = s["h"].double()
        y = h[:, :c] * torch.sigmoid(h[:, :c]) * h[:, c:]
        out = {"y": y, "amax": y.to(TYPES[kind]).double().abs().max().view(1)}
        if op == "swiglu_step":
            h = _exact_rounded(s["h"], case["saved"])
            gate, up, dy = h[:, :c], h[:, c:], s["dy"].double()
            sig = torch.sigmoid(gate)
            out["dh"] = torch.cat([dy * up * (sig + gate * sig * (1 - sig)), dy * gate * sig], dim=1)
        return out
    if op == "wgrad":
        x = _exact_saved(s["codes"], s["scales"], case["saved"])
        if s["row_index"] is not None:
            x = x[s["row_index"].long()]
        at = s["offsets"].tolist()
        dw = [s["dy"][a:b].double().t() @ x[a:b] for a, b in zip(at, at[1:])]
        return {"dw": torch.cat(dw)}
    t, k, c = case["tokens"], case["topk"], case["cols"]
    slot, w = s["slot_row"].long(), s["weights"].double()
    if op == "combine":
        out = torch.zeros(t, c, dtype=torch.float64, device=DEVICE)
        for j in range(k):
            out += w[:, j:j + 1] * s["rows"][slot[:, j]].double()
        return {"out": out}
    d_out = s["d_out"].double()
    d_rows = torch.zeros(t * k, c, dtype=torch.float64, device=DEVICE)
    d_weights = torch.zeros(t, k, dtype=torch.float64, device=DEVICE)
    for j in range(k):
        d_rows[slot[:, j]] = w[:, j:j + 1] * d_out
        d_weights[:, j] = (d_out * s["rows"][slot[:, j]].double()).sum(1)
    return {"d_rows": d_rows, "d_weights": d_weights}
