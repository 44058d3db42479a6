"""The dense layer's operators on matrices whose offsets pass 32 bits: samples near
both ends against the formula, which small tests check in full."""
import numpy as np
import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

SEED, COUNTER = 77, 2 ** 40


def test_linear_with_many_results():
    """2^32 + elements of z and out, from one block of K."""
    M, N, K = 65536 + 70, 65536 + 24, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-4, 5, (M, K), generator=g, device=dev()).to(torch.bfloat16)
    w = torch.randint(-4, 5, (N, K), generator=g, device=dev()).float()
    W = mx.mx_quantize(w, mx.empty(mx.FORMATS["mxint8"], N, K, dev()))  # (exact)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=dev())
    z = torch.empty_like(out)
    mx.mx_linear(x, W, out, act=mx.MX_ACT_RELU, z=z, drop=0.5, seed=SEED, counter=COUNTER)
    per = -(-N // 8)
    for r in (0, 1, 32768, M - 66, M - 1):
        want = x[r].float() @ w.t()  # whole numbers below 2^10
        assert torch.equal(z[r], want.to(torch.bfloat16)), r
        fac = torch.from_numpy(R.drop_factors(0.5, SEED, COUNTER + r * per, 1, N)[0]).to(dev())
        assert torch.equal(out[r].double(), (want.clamp(min=0) * fac).to(torch.bfloat16).double()), r


@pytest.mark.parametrize("M", [2, 20, 70])
def test_linear_with_many_weights(M):
    """codes past 2^32 bytes"""
    N, K = 2 ** 19 + 40, 16384
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    scales = torch.randint(120, 124, (N, K // 32), generator=g, device=dev(), dtype=torch.uint8)
    x = torch.randn(M, K, generator=g, device=dev()).to(torch.bfloat16)
    out = torch.empty(M, N, device=dev())
    mx.mx_linear(x, mx.MXTensor(mx.FORMATS["mxfp4"], N, K, codes, scales), out)
    for a in (0, 2 ** 18 - 3, N - 9):
        rows = slice(a, a + 9)
        w = R.weights("mxfp4", codes[rows].cpu().numpy(), scales[rows].cpu().numpy())
        x64 = x.double().cpu().numpy()
        want, tol = x64 @ w.T, 1e-5 * (np.abs(x64) @ np.abs(w).T)
        assert (np.abs(out[:, rows].double().cpu().numpy() - want) <= tol).all(), a


def test_dropout_and_epilogue_backward():
    rows, cols = 2 ** 17 + 3, 2 ** 15 + 8
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device=dev())
    per = cols // 8
    out = torch.empty_like(x)
    mx.mx_dropout(x, out, 0.25, SEED, COUNTER)
    some = (0, 65535, 65536, rows - 1)
    masks = {r: torch.from_numpy(R.drop_factors(0.25, SEED, COUNTER + r * per, 1, cols)[0]).to(dev()) for r in some}
    for r in some:
        assert torch.equal(out[r], masks[r].to(torch.bfloat16)), r
    d_bias = torch.empty(cols, device=dev())
    mx.mx_epilogue_backward(x, x, out, d_bias, act=mx.MX_ACT_RELU, drop=0.25, seed=SEED, counter=COUNTER)
    for r in some:
        assert torch.equal(out[r], masks[r].to(torch.bfloat16)), r
    # a column keeps rows * 0.75 of its ones: eight standard deviations (7 per 32768 columns), and the sums' rounding
    kept = d_bias.double() * 0.75
    assert ((kept - rows * 0.75).abs() <= 8 * (rows * 0.1875) ** 0.5 + rows * rows * 2.0 ** -24 / 64).all()


@pytest.mark.parametrize("rows", [0, 1])
def test_bias_gradient_of_many_columns(rows):
    cols = 2 ** 28 + 24
    d_out = torch.full((rows, cols), 0.5, dtype=torch.bfloat16, device=dev())
    d_bias = torch.full((cols,), 7.0, device=dev())
    mx.mx_epilogue_backward(d_out, None, None, d_bias)
    assert (d_bias == 0.5 * rows).all()
