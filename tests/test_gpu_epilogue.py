"""mx_dropout and mx_epilogue_backward against their formulas in 64 bits."""
import numpy as np
import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev
    from tests.test_gpu_linear import check, matrix

SEED, COUNTER = 2 ** 63 + 11, 2 ** 34 + 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (1, 8, 0, 0), (3, 13, 0, 0), (5, 64, 0, 0), (7, 100, 4, 0),
                                                 (33, 257, 8, 8), (200, 520, 3, 1), (1000, 24, 0, 0)])
@pytest.mark.parametrize("drop", [0.0, 0.1, 0.5, 0.99999])
def test_dropout(dtype, rows, cols, pad, shift, drop):
    g = np.random.default_rng(rows + cols)
    x, x64 = matrix(g.normal(size=(rows, cols)), dtype, pad, shift)
    r, r64 = matrix(g.normal(size=(rows, cols)), dtype, pad)
    fac = R.drop_factors(drop, SEED, COUNTER, rows, cols)
    h = R.HALF_STEP[dtype]
    want = x64 * fac
    tol = 2 * R.U * np.abs(want)
    out = matrix(np.zeros((rows, cols)), dtype, pad, shift)[0]
    mx.mx_dropout(x, out, drop, SEED, COUNTER)
    check(out, want, tol + h * (np.abs(want) + tol), "plain")
    assert ((out.double().cpu().numpy() == 0) == (want == 0)).all()
    if pad:
        assert (out.as_strided((rows, pad), (cols + pad, 1), shift + cols) == 99).all()
    w2 = want + r64
    tol = tol + R.U * (np.abs(w2) + tol)
    tol = tol + h * (np.abs(w2) + tol)
    mx.mx_dropout(x, out, drop, SEED, COUNTER, residual=r)
    check(out, w2, tol, "residual")
    mx.mx_dropout(x, r, drop, SEED, COUNTER, residual=r)  # in place of the residual
    check(r, w2, tol, "residual in place")
    mx.mx_dropout(x, x, drop, SEED, COUNTER)
    check(x, want, 2 * R.U * np.abs(want) + 1.01 * h * np.abs(want), "in place")


def test_dropped_values_are_zero_whatever_they_were():
    x = torch.full((4, 64), float("nan"), device=dev())
    out = mx.mx_dropout(x, torch.empty_like(x), 0.5, SEED, COUNTER)
    dropped = torch.from_numpy(R.drop_factors(0.5, SEED, COUNTER, 4, 64) == 0).to(dev())
    assert (out[dropped] == 0).all() and torch.isnan(out[~dropped]).all()


def test_gradient_of_dropout_is_the_same_call():
    """<d, drop(x)> is linear in x: differences of it are exact."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, d = (torch.randint(-8, 9, (6, 40), generator=g, device=dev()).float() for _ in range(2))
    dx = mx.mx_dropout(d, torch.empty_like(d), 0.5, 3, 4)
    for i in range(0, 240, 7):
        up = x.clone()
        up.view(-1)[i] += 1
        a, b = (mx.mx_dropout(v, torch.empty_like(v), 0.5, 3, 4) for v in (up, x))
        assert float((d * (a - b)).sum()) == float(dx.view(-1)[i])


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (2, 9, 0, 0), (17, 64, 0, 0), (100, 333, 3, 1),
                                                 (700, 40, 8, 8), (3, 4100, 0, 0), (1025, 520, 0, 0)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_epilogue_backward(act, dtype, rows, cols, pad, shift, drop):
    g = np.random.default_rng(rows * 7 + cols)
    d, d64 = matrix(g.normal(size=(rows, cols)), dtype, pad, shift)
    z, z64 = matrix(g.normal(size=(rows, cols)) * 3, dtype, pad)
    fac = R.drop_factors(drop, SEED, COUNTER, rows, cols) if drop else None
    (want, tol), (bw, bt) = R.epilogue_backward(d64, z64, act, fac, dtype)
    dz = matrix(np.zeros((rows, cols)), dtype, pad, shift)[0]
    db = torch.full((cols,), 5.0, device=dev())
    kw = dict(act=mx.ACTIVATIONS[act], drop=drop, seed=SEED, counter=COUNTER)
    mx.mx_epilogue_backward(d, z, dz, db, **kw)
    check(dz, want, tol, "d_z")
    check(db, bw, bt, "d_bias")
    first, bias = dz.clone(), db.clone()
    ws = torch.full((mx.mx_epilogue_workspace_bytes(rows, cols),), 255, dtype=torch.uint8, device=dev())
    db.fill_(7)
    mx.mx_epilogue_backward(d, z, None, db, workspace=ws, **kw)  # each alone
    assert torch.equal(db, bias)
    mx.mx_epilogue_backward(d, z, z, **kw)  # in place of z
    assert torch.equal(z, first)
    z.copy_(torch.from_numpy(z64))
    mx.mx_epilogue_backward(d, z if act != "none" else None, d, db, **kw)  # in place of d_out
    assert torch.equal(d, first) and torch.equal(db, bias)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(127, 4), (128, 65), (128, 2051), (129, 2051), (129, 4)])
def test_few_rows(dtype, rows, cols):
    g = np.random.default_rng(rows + cols)
    d, d64 = matrix(g.normal(size=(rows, cols)), dtype)
    z, z64 = matrix(g.normal(size=(rows, cols)), dtype)
    (want, tol), (bw, bt) = R.epilogue_backward(d64, z64, "silu", R.drop_factors(0.3, SEED, COUNTER, rows, cols), dtype)
    dz, db = torch.empty_like(d), torch.full((cols,), 5.0, device=dev())
    mx.mx_epilogue_backward(d, z, dz, db, act=mx.MX_ACT_SILU, drop=0.3, seed=SEED, counter=COUNTER)
    check(dz, want, tol, "d_z")
    check(db, bw, bt, "d_bias")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_far_arguments(act):
    """The whole range of finite z: slopes of 0 and 1 at its ends, no NaN."""
    z64 = np.concatenate([np.linspace(-100, 100, 4001), [-3e38, -1e20, 1e20, 3e38, 0.0, -0.0]])[None]
    z, z64 = matrix(z64, "f32")
    one = torch.ones_like(z)
    dz, out = torch.empty_like(z), torch.empty_like(z)
    mx.mx_epilogue_backward(one, z, dz, act=mx.ACTIVATIONS[act])
    with np.errstate(over="ignore", invalid="ignore"):
        (want, tol), _ = R.epilogue_backward(np.ones_like(z64[:, :4001]), z64[:, :4001], act, None, "f32")
    check(dz[:, :4001], want, tol, act)
    assert dz[0, 4001:].tolist() == pytest.approx([0, 0, 1, 1, 0.5, 0.5], abs=20 * R.U)
    # the values, through a product with nothing to sum: z is the bias
    W = mx.empty(mx.FORMATS["mxfp8"], z.shape[1], 0, dev())
    mx.mx_linear(torch.empty(1, 0, dtype=torch.bfloat16, device=dev()), W, out, bias=z[0].contiguous(),
                 act=mx.ACTIVATIONS[act])
    y, tol = R.act(z64[:, :4001], act)
    check(out[:, :4001], y, tol, act)
    assert out[0, 4003:].tolist() == z[0, 4003:].tolist() and (out[0, 4001:4003] == 0).all()


def test_empty():
    e = torch.empty(0, 24, device=dev())
    db = torch.full((24,), 3.0, device=dev())
    mx.mx_epilogue_backward(e, e, e.clone(), db, act=mx.MX_ACT_SILU)
    assert (db == 0).all()
    mx.mx_dropout(e, e.clone(), 0.5)


def test_another_stream():
    g = torch.Generator(device="cuda").manual_seed(2)
    d, z = (torch.randn(3000, 264, generator=g, device=dev()) for _ in range(2))
    want, wb = mx.mx_epilogue_backward(d, z, torch.empty_like(d), torch.empty(264, device=dev()), act=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, gb = mx.mx_epilogue_backward(d, z, torch.empty_like(d), torch.empty(264, device=dev()), act=2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(wb, gb)
