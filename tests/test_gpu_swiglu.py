"""The gated activation and its backward pass from an 8-bit checkpoint, against
their 64-bit definitions.

Bounds (u = 2^-24): the sigmoid's argument is rounded twice and the exponential
and the reciprocal are good to one unit, so s has relative error
E_S = u (8 + 4 |gate|); products add u each.  1 - s has absolute error
s E_S + u, which gate multiplies.  Below 2^-126 exponentials may vanish."""
import numpy as np
import pytest
import torch

from tests import moe_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FMT = ["mxfp8", "mxfp8_e5m2", "mxint8"]


def matrix(x, kind, pad=0):
    t = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=DT[kind], device=dev())
    t[:, : x.shape[1]] = torch.from_numpy(x.astype(np.float32)).to(dev())
    return t[:, : x.shape[1]]


def act(rows, cols, seed):
    g = np.random.default_rng([seed, rows, cols])
    x = g.standard_normal((rows, cols)) * 2
    return x * np.where(g.random(cols) < 0.05, 12.0, 1.0)


def host(t):
    return t.detach().cpu().double().numpy()


def check_y(y, h, kind):
    c = h.shape[1] // 2
    want = moe_ref.swiglu(h)
    tol = U * (12 + 4 * np.abs(h[:, :c])) * np.abs(want) + 1e-36 * (1 + np.abs(h[:, c:]))
    if kind == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(host(y) - want) <= tol)


def decoded(saved):
    out = torch.empty(saved.rows, saved.cols, device=dev())
    mx.mx_dequantize(saved, out)
    return host(out)


def check_dh(dh, h, dy, kind):
    c = h.shape[1] // 2
    g, u = h[:, :c], h[:, c:]
    s = moe_ref.sigmoid(g)
    want = moe_ref.swiglu_backward(h, dy)
    es = U * (8 + 4 * np.abs(g))
    tol_g = np.abs(dy * u) * (s * es * (1 + np.abs(g)) * 2 + s * np.abs(g) * (s * es + U) + 8 * U * s * (1 + np.abs(g)))
    tol_u = np.abs(dy * g) * s * (es + 4 * U)
    tol = np.concatenate([tol_g, tol_u], axis=1) + 1e-36 * np.abs(np.concatenate([dy * u, dy * g], axis=1)) + 1e-37
    if kind == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(host(dh) - want) <= tol)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (8, 2048), (3, 96), (33, 160), (257, 64), (130, 1056)])
def test_forward_without_a_checkpoint(rows, cols, kind):
    for pad in (0, 8):
        h = matrix(act(rows, 2 * cols, 1), kind, pad)
        y = matrix(np.zeros((rows, cols)), kind, pad)
        amax = torch.full((1,), -5.0, device=dev())
        mx.mx_swiglu(h, y, amax=amax)
        torch.cuda.synchronize()
        check_y(y, host(h), kind)
        assert float(amax) == float(y.float().abs().max())
        if pad:
            assert bool((y._base[:, cols:] == 7.0).all())


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rnd", ["rne", "sr"])
@pytest.mark.parametrize("rows,cols,kind", [(1, 32, "bf16"), (37, 96, "f32"), (64, 544, "bf16"), (301, 64, "f32")])
def test_checkpoint_is_the_quantizers_and_backward_reads_it(rows, cols, kind, rnd, fmt):
    h = matrix(act(rows, 2 * cols, 2), kind, 8)
    saved, plain = (mx.empty(mx.FORMATS[fmt], rows, 2 * cols, dev()) for _ in range(2))
    y = matrix(np.zeros((rows, cols)), kind)
    how = dict(rnd=mx.MX_SR if rnd == "sr" else mx.MX_RNE, seed=5, counter=11)
    mx.mx_swiglu(h, y, saved=saved, **how)
    mx.mx_quantize(h, plain, **how)
    torch.cuda.synchronize()
    check_y(y, host(h), kind)
    assert torch.equal(saved.codes, plain.codes) and torch.equal(saved.scales, plain.scales)
    g = np.random.default_rng(3)
    dy = matrix(g.standard_normal((rows, cols)) * 0.1, kind, 8)
    dh = matrix(np.zeros((rows, 2 * cols)), kind, 8)
    ys = mx.empty(mx.FORMATS[fmt], rows, cols, dev())
    mx.mx_swiglu_backward(saved, dy, dh, y_saved=ys)
    torch.cuda.synchronize()
    hd = decoded(saved)
    check_dh(dh, hd, host(dy), kind)
    assert bool((dh._base[:, 2 * cols:] == 7.0).all())
    # y of the decoded values, to within the format's step at the block's
    # largest value: E4M3 2^-4, E5M2 2^-3, INT8 2^-7 of it (half a step), or
    # saturation of E4M3 (448 of up to 512) and of E5M2
    want = moe_ref.swiglu(hd)
    blocks = np.abs(want).reshape(rows, cols // 32, 32).max(2).repeat(32, axis=1)
    part = {"mxfp8": 2.0 ** -3, "mxfp8_e5m2": 2.0 ** -2, "mxint8": 2.0 ** -6}[fmt]
    assert np.all(np.abs(decoded(ys) - want) <= part * blocks + 1e-30)
    only = matrix(np.zeros((rows, 2 * cols)), kind, 8)
    mx.mx_swiglu_backward(saved, dy, only)
    torch.cuda.synchronize()
    assert torch.equal(only, dh)


@pytest.mark.parametrize("fmt", FMT)
def test_recomputed_activation_is_quantized_as_the_quantizer_does(fmt):
    """FP32: the recomputed y is the forward kernel's y of the decoded values,
    so its codes are the quantizer's of that."""
    rows, cols = 65, 192
    saved = mx.empty(mx.FORMATS[fmt], rows, 2 * cols, dev())
    mx.mx_quantize(matrix(act(rows, 2 * cols, 4), "f32"), saved)
    hd = torch.empty(rows, 2 * cols, device=dev())
    mx.mx_dequantize(saved, hd)
    y, want, ys = torch.empty(rows, cols, device=dev()), mx.empty(mx.FORMATS[fmt], rows, cols, dev()), mx.empty(
        mx.FORMATS[fmt], rows, cols, dev())
    mx.mx_swiglu(hd, y)
    mx.mx_quantize(y, want)
    dh = torch.empty(rows, 2 * cols, device=dev())
    mx.mx_swiglu_backward(saved, torch.ones(rows, cols, device=dev()), dh, y_saved=ys)
    torch.cuda.synchronize()
    assert torch.equal(ys.codes, want.codes) and torch.equal(ys.scales, want.scales)


def test_extreme_gates():
    h = np.zeros((2, 128))
    h[0, :8] = [0.0, -0.0, 88.0, -88.0, 200.0, -200.0, 1e4, -1e4]
    h[0, 64:72] = 3.0
    h[1, :4] = [3e38, -3e38, 1e-38, -1e-38]
    h[1, 64:68] = 1e-30
    for kind in DT:
        t = matrix(h, kind)
        y = matrix(np.zeros((2, 64)), kind)
        mx.mx_swiglu(t, y)
        torch.cuda.synchronize()
        check_y(y, host(t), kind)
        assert bool(torch.isfinite(y).all())


def test_nan_block_stays_in_its_block():
    rows, cols = 4, 64
    x = act(rows, 2 * cols, 5)
    x[1, 3] = np.nan
    x[2, cols + 40] = np.inf
    h = matrix(x, "f32")
    saved = mx.empty(mx.MX_MXFP8_E4M3, rows, 2 * cols, dev())
    y = torch.empty(rows, cols, device=dev())
    mx.mx_swiglu(h, y, saved=saved)
    dh = torch.empty(rows, 2 * cols, device=dev())
    mx.mx_swiglu_backward(saved, torch.ones(rows, cols, device=dev()), dh)
    torch.cuda.synchronize()
    bad = torch.isnan(dh).cpu().numpy()
    want = np.zeros_like(bad)
    want[1, 0:32] = want[1, cols:cols + 32] = True         # the gate's block feeds both gradients
    want[2, 32:64] = True                                   # the up block only the gate's
    assert np.array_equal(bad, want)


def test_gradient_against_differences():
    """The kernel's dh for an exactly representable h against central
    differences of the 64-bit y: truncation h^2 / 6 * |third derivative| < 1e-9
    at h = 1e-4, FP32 1e-6 of values below 10."""
    rows, cols = 2, 32
    x = np.round(act(rows, 2 * cols, 6).clip(-3, 3) * 4) / 4
    x[:, 0] = 3.0                        # the largest of its block: E4M3 holds quarters up to 3.75 exactly
    x[:, cols] = 3.0
    saved = mx.empty(mx.MX_MXINT8, rows, 2 * cols, dev())
    mx.mx_quantize(matrix(x, "f32"), saved)
    assert np.array_equal(decoded(saved), x)
    dy = np.random.default_rng(7).standard_normal((rows, cols)).astype(np.float32).astype(np.float64)
    dh = torch.empty(rows, 2 * cols, device=dev())
    mx.mx_swiglu_backward(saved, matrix(dy, "f32"), dh)
    got, h = host(dh), 1e-4
    for r in range(rows):
        for c in range(2 * cols):
            a, b = x.copy(), x.copy()
            a[r, c] += h
            b[r, c] -= h
            quot = ((moe_ref.swiglu(a) - moe_ref.swiglu(b)) * dy).sum() / (2 * h)
            assert abs(got[r, c] - quot) <= 2e-5


def test_empty():
    for rows, cols in ((0, 64), (5, 0)):
        amax = torch.full((1,), 3.0, device=dev())
        mx.mx_swiglu(torch.empty(rows, 2 * cols, device=dev()), torch.empty(rows, cols, device=dev()), amax=amax)
        torch.cuda.synchronize()
        assert float(amax) == 0.0
