"""The library's calls on the measured cases of a dense layer and of token scoring and
on cases drawn from the same ranges, against the 64-bit definitions of
perf/more_operators.py: every element within the bounds of dense_bounds.py."""
import random

import pytest
import torch

from perf import more_operators as P
from tests import dense_bounds as D
from tests.linear_shapes import SHAPES

pytestmark = pytest.mark.gpu


def within(got, want, tol, what):
    got = got.double()
    ok = ((got - want).abs() <= tol) | (got == want) | (got.isnan() & want.isnan())
    bad = (~ok).nonzero()[:4].tolist()
    assert not bad, (what, int((~ok).sum()), [(i, float(got[tuple(i)]), float(want[tuple(i)]), float(tol[tuple(i)]))
                                              for i in bad])


def check(case, seed, monkeypatch):
    monkeypatch.setattr(P, "own", True)
    s = P.prepare(case, seed)
    got = P.run(s)
    torch.cuda.synchronize()
    op = case["op"]
    if op == "linear":
        fac = P._exact_factors(s["stream"], case["rows"], case["n"], case["drop"]) if case["drop"] else None
        opt = lambda t: None if t is None else t.double()
        want = D.linear(case, s["x"].double(), P._exact_weights(s), opt(s["bias"]), fac, opt(s["residual"]))
        for n in got:
            within(got[n], *want[n], n)
        return
    if op == "dropout":
        want = P.exact(case, seed)["out"]
        # the factor, its product and the sum in FP32
        r = 0 if s["residual"] is None else s["residual"].double()
        e = 2 * D.U * (want - r).abs() + D.U * want.abs()
        return within(got["out"], want, D.stored(want, e, case["type"]), "out")
    if op == "epilogue_backward":
        want = P.exact(case, seed)
        fac = P._exact_factors(s["stream"], case["rows"], case["cols"], case["drop"]) if case["drop"] else None
        tol = D.epilogue_backward(case, s["d_out"].double(), s["z"].double(), fac, want)
        for n in got:
            within(got[n], want[n], tol[n], n)
        return
    want, there = P.exact(case, seed), s["target"] >= 0
    for a in range(0, case["tokens"], 512):  # (a part of the rows at a time)
        rows = slice(a, a + 512)
        x, target, ok = s["logits"][rows].double(), s["target"][rows], there[rows]
        if op == "logprob_backward":
            tol = D.logprob_backward(case, x, target, s["d_logp"][rows].double(), s["d_entropy"][rows].double(),
                                     want["d_logits"][rows])
            within(got["d_logits"][rows], want["d_logits"][rows], tol, "d_logits")
            continue
        d, log_sum, e, entropy, e_entropy = D.scores(x, case["scale"])
        one = lambda v: torch.where(ok, v, 0.0)
        at = target.clamp(min=0)[:, None]
        e_logp = D.log_probability(d.gather(1, at)[:, 0], log_sum, e)
        for n, tol in (("logp", e_logp), ("row_max", 0 * e), ("log_sum", e), ("entropy", e_entropy)):
            within(got[n][rows], want[n][rows], one(tol), n)
        if case["topk"]:
            ids = want["top_id"][rows]
            assert torch.equal(got["top_id"][rows], ids)
            tol = D.log_probability(d.gather(1, ids.long()), log_sum[:, None], e[:, None])
            within(got["top_logp"][rows], want["top_logp"][rows], tol, "top_logp")


@pytest.mark.parametrize("case", P.listed(), ids=lambda c: c["name"])
def test_listed(case, monkeypatch):
    check(case, 3, monkeypatch)


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed, monkeypatch):
    case = P.draw(random.Random(1000 + seed))
    print(case, flush=True)
    check(case, seed, monkeypatch)


# Every kernel of the product with every format and every part of an epilogue: whole
# steps of K, a remainder alone, both, long sums.
EPILOGUES = [("none", False, 0.0, True), ("gelu", True, 0.0, False), ("silu", False, 0.1, True),
             ("gelu_tanh", True, 0.5, True), ("relu", True, 0.1, False), ("none", True, 0.0, True),
             ("gelu", False, 0.1, True)]


@pytest.mark.parametrize("weights", P.WEIGHTS)
@pytest.mark.parametrize("k", [96, 128, 160, 1056, 2048])
@pytest.mark.parametrize("kernel", SHAPES)
def test_linear_kernels(kernel, k, weights, monkeypatch):
    n = P.WEIGHTS.index(weights) + 3 * k // 32
    for i, (rows, cols) in enumerate(SHAPES[kernel]):
        act, keep_z, drop, residual = EPILOGUES[(n + 2 * i) % len(EPILOGUES)]
        case = {"op": "linear", "rows": rows, "n": cols, "k": k, "weights": weights, "type": ("bf16", "f32")[(n + i) % 2],
                "bias": ("bf16", "f32", "none")[(n + i) % 3], "act": act, "keep_z": keep_z, "drop": drop,
                "residual": residual}
        print(case, flush=True)
        check(case, n + i, monkeypatch)
