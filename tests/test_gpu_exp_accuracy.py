"""Softmax weights, gradients of scores and the gated activation far from 0:
the exponential's error does not grow with its argument.

Bounds (u = 2^-24).  The hardware's 2^x is good to one unit in the last place
(2 u); it gets x = d log2(e) as rounded, and e^d = 2^x (1 + (d - x ln 2)), whose
bracket is exact to far below u, adds u: 3 u.  All scores here are multiples of
1/8 below 128, so differences of them are exact.
  p = e / sum:  e 3 u, the sum 3 u and u for each of at most VPL + 5 adds of
  positive terms (VPL scores a lane), 1 / sum and the product u each:
  E_P = u (13 + VPL).
  d_x = q d_w - p <q, d_w> (no loss): p and q within E_P, the sum over the slots
  4 u more, three roundings: (2 E_P + 8 u) of the terms' sizes.
  sigmoid = 1 / (1 + e^-g): e 3 u, the sum u, the quotient u after one Newton
  step: 5 u.  y: two products more, 7 u.  d_up the same.  d_gate = dy up s inner,
  inner = 1 + g (1 - s): inner is off by |g| (5 u s + u (1 - s)) + u |inner|, and
  s and three products add 8 u."""
import numpy as np
import pytest
import torch

from tests import moe_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

U = 2.0 ** -24


def host(t):
    return t.detach().cpu().double().numpy()


def vpl(E):
    return next(v for n, v in ((16, 1), (32, 2), (64, 4), (128, 8), (256, 16), (512, 8), (1024, 16)) if E <= n)


def scores(T, E, seed):
    """Multiples of 1/8 from -40 to 40, the whole width in every row."""
    g = np.random.default_rng([seed, T, E])
    x = g.integers(-320, 321, (T, E)) / 8.0
    for t in range(T):
        x[t, g.permutation(E)[:2]] = 40.0, -40.0
    return torch.from_numpy(x.astype(np.float32)).to(dev())


def route(x, topk, normalize):
    r = mx.routing(x.shape[0], x.shape[1], topk, device=dev())
    mx.mx_route(x, r, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("E", [5, 16, 32, 60, 128, 256, 500, 1024])
def test_probabilities(E):
    ep = U * (13 + vpl(E))
    for t in range(20):  # one token: the sums over the tokens are its probabilities
        x = scores(1, E, t)
        r = route(x, 1, False)
        p = moe_ref.route(host(x), 1)["p"][0]
        assert np.all(np.abs(host(r.prob_sum) - p) <= ep * p + 1e-37), float(np.max(np.abs(host(r.prob_sum) - p) / p / U))


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("E,topk", [(5, 5), (16, 16), (32, 16), (300, 16)])
def test_weights_and_their_gradient(E, topk, normalize):
    T = 100
    x = scores(T, E, 1)
    r = route(x, topk, normalize)
    want = moe_ref.route(host(x), topk, normalize=normalize)
    assert np.array_equal(host(r.experts), want["experts"])
    ep = U * (13 + vpl(E))
    w = want["weights"]
    assert np.all(np.abs(host(r.weights) - w) <= ep * w + 1e-37)
    dw = torch.from_numpy(np.random.default_rng(2).standard_normal((T, topk)).astype(np.float32)).to(dev())
    d = torch.empty_like(x)
    mx.mx_route_backward(x, r, dw, None, d, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    torch.cuda.synchronize()
    dx, size = moe_ref.route_backward(want["p"], want["experts"], want["counts"], T, host(dw), 0.0, normalize)
    assert np.all(np.abs(host(d) - dx) <= (2 * ep + 8 * U) * size + 1e-37)


def gates(rows, cols, seed):
    """[gate | up], gates from -80 to 80 (e^80 and its inverse are FP32 numbers)."""
    g = np.random.default_rng([seed, rows, cols])
    gate = g.uniform(-80, 80, (rows, cols)) * np.where(g.random((rows, cols)) < 0.5, 1.0, 0.05)
    return np.concatenate([gate, g.standard_normal((rows, cols))], axis=1).astype(np.float32)


def test_activation():
    rows, cols = 200, 256
    h = gates(rows, cols, 3)
    y = torch.empty(rows, cols, device=dev())
    mx.mx_swiglu(torch.from_numpy(h).to(dev()), y)
    torch.cuda.synchronize()
    want = moe_ref.swiglu(h.astype(np.float64))
    assert np.all(np.abs(host(y) - want) <= 8 * U * np.abs(want)), float(np.max(np.abs(host(y) - want) / np.abs(want) / U))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp8_e5m2", "mxint8"])
def test_activation_backward(fmt):
    rows, cols = 200, 256
    saved = mx.empty(mx.FORMATS[fmt], rows, 2 * cols, dev())
    mx.mx_quantize(torch.from_numpy(gates(rows, cols, 4)).to(dev()), saved)
    h = torch.empty(rows, 2 * cols, device=dev())
    mx.mx_dequantize(saved, h)
    dy = torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(5), device=dev())
    dh = torch.empty(rows, 2 * cols, device=dev())
    mx.mx_swiglu_backward(saved, dy, dh)
    torch.cuda.synchronize()
    h, d = host(h), host(dy)
    assert np.abs(h[:, :cols]).max() <= 80
    g, u = h[:, :cols], h[:, cols:]
    s = moe_ref.sigmoid(g)
    inner, rest = 1 + g * (1 - s), moe_ref.sigmoid(-g)
    tol_gate = U * np.abs(d * u) * s * (np.abs(g) * (5 * s + rest) + 10 * np.abs(inner))
    tol_up = 8 * U * np.abs(d * g) * s
    tol = np.concatenate([tol_gate, tol_up], axis=1) + 1e-37
    assert np.all(np.abs(host(dh) - moe_ref.swiglu_backward(h, d)) <= tol)
