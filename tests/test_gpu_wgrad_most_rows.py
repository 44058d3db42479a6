"""The weight gradient of as many rows as the call takes (2^31 - 1): the rows
before, at and past every 64th part of the range are summed.  dY is zero but for
a few rows, whose products are small integers, so the sums are exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev


def test_all_rows_count():
    R, N, K, x_rows = (1 << 31) - 1, 8, 32, 8
    assert mx.mx_wgrad_workspace_bytes(R, N, K, 1) > 0  # summed in parts
    x = (torch.arange(x_rows * K, device=dev()).view(x_rows, K) % 13 - 6).float()
    X = mx.empty(mx.MX_MXFP8_E4M3, x_rows, K, dev())
    mx.mx_quantize(x, X)
    back = torch.empty_like(x)
    mx.mx_dequantize(X, back)
    assert torch.equal(back, x)
    at = sorted({min(max(i * (R // 64) + d, 0), R - 1) for i in range(65) for d in (-1, 0, 1)} | {191, 192, R - 64})
    at = torch.tensor(at, device=dev())
    some = (torch.arange(len(at) * N, device=dev()).view(-1, N) % 7 - 3).to(torch.bfloat16)
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device=dev())
    dy[at] = some
    index = torch.zeros(R, dtype=torch.int32, device=dev())
    src = torch.arange(len(at), device=dev()) % x_rows
    index[at] = src.int()
    dw = torch.full((N, K), 7.0, device=dev())
    mx.mx_wgrad_grouped(dy, X, index, 1, None, dw)
    torch.cuda.synchronize()
    assert torch.equal(dw.double(), some.double().t() @ x[src].double())
