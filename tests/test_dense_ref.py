"""The 64-bit definitions that the dense layer's GPU tests compare with: their
gradients against differences, their random stream against the oracle's, their
weights against the oracle's decoder."""
import numpy as np
import pytest

from tests import dense_ref as R


def differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_epilogue_gradient(kind):
    g = np.random.default_rng(3)
    z, d = g.normal(size=(5, 9)) * 2, g.normal(size=(5, 9))
    fac = R.drop_factors(0.3, 5, 7, 5, 9)
    f = lambda v: (d * R.act(v, kind)[0] * fac).sum()
    (dz, _), (db, _) = R.epilogue_backward(d, z, kind, fac, "f32")
    np.testing.assert_allclose(dz, differences(f, z), rtol=1e-6, atol=1e-8)
    by_bias = differences(lambda b: f(z + b), np.zeros(9))
    np.testing.assert_allclose(db, by_bias, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_logprob_gradient(scale):
    g = np.random.default_rng(4)
    x, target = g.normal(size=(4, 11)) * 3, np.array([0, 10, -1, 5])
    dl, dh = g.normal(size=4), g.normal(size=4)

    def f(v):
        o, _ = R.logprob(v, target, scale, 0)
        return (dl * o["logp"] + dh * o["entropy"]).sum()

    _, tol = R.logprob(x, target, scale, 0)
    d, _ = R.logprob_backward(x, target, scale, dl, dh, tol, "f32")
    np.testing.assert_allclose(d, differences(f, x), rtol=1e-5, atol=1e-8)


def test_draws_are_the_quantizers_stream(orc):
    for cols in (8, 16, 24):
        d = R.draws(2 ** 40 + 17, 2 ** 33 - 1, 3, cols)
        for r in range(3):
            for c in range(cols):
                assert d[r, c] == orc.rand16(2 ** 40 + 17, 2 ** 33 - 1, r * cols + c)
    # a row of another length starts at a block of its own
    d = R.draws(9, 4, 3, 13)
    assert [d[2, c] for c in (0, 12)] == [orc.rand16(9, 4, 32), orc.rand16(9, 4, 44)]


def test_drop_rate():
    f = R.drop_factors(0.1, 1, 0, 400, 401)
    assert set(np.unique(f)) == {0.0, 65536 / (65536 - 6554)}
    n = f.size  # five standard deviations
    assert abs((f == 0).mean() - 6554 / 65536) < 5 * (0.09 / n) ** 0.5


@pytest.mark.parametrize("name,fmt", [("mxfp8", 1), ("mxfp4", 2), ("nvfp4", 3), ("mxint8", 4), ("mxfp8_e5m2", 5)])
def test_weights_against_the_oracle(orc, name, fmt):
    g = np.random.default_rng(fmt)
    x = g.normal(size=(6, 96)).astype(np.float32)
    q = orc.quantize(x, fmt)
    codes, scales = q[0], q[1]
    ts = float(q[2]) if fmt == 3 else 1.0
    want = orc.dequantize(fmt, codes, scales, ts if fmt == 3 else None, 6, 96)
    got = R.weights(name, np.asarray(codes).reshape(6, -1), np.asarray(scales).reshape(6, -1), ts)
    np.testing.assert_allclose(got, want, rtol=1.2e-7, atol=0)
