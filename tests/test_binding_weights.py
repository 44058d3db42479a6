"""What mx_linear's binding asks of the weights' tensors: dense bytes of the weights'
size, since the library cannot see how long they are."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def mx():
    import microscaling_precision_gemm_amd as mx
    if not os.path.exists(mx.LIB_PATH):
        from microscaling_precision_gemm_amd.build import build
        build()
    mx.load()
    return mx


SIZES = {"mxfp4": (32, 2), "nvfp4": (32, 4), "mxfp8": (64, 2), "mxfp8_e5m2": (64, 2), "mxint8": (64, 2)}  # a row of 64


@pytest.mark.parametrize("fmt", SIZES)
def test_tensors_of_another_size_type_or_order_are_refused(mx, fmt):
    c, s = SIZES[fmt]
    z = lambda *shape, dt=torch.uint8: torch.zeros(*shape, dtype=dt)
    ts = torch.ones(1) if fmt == "nvfp4" else None
    bad = [(z(8, c - 1), z(8, s), ts), (z(7, c), z(8, s), ts), (z(8, c + 16), z(8, s), ts), (z(0), z(8, s), ts),
           (z(8, c), z(8, s - 1), ts), (z(8, c), z(7, s), ts), (z(8, c), z(0), ts),
           (z(c, 8).t(), z(8, s), ts), (z(8, c), z(s, 8).t(), ts), (z(8, 2 * c)[:, ::2], z(8, s), ts),
           (z(8, 2 * c)[:, :c], z(8, s), ts), (z(1, c).expand(8, c), z(8, s), ts),
           (z(8, c, dt=torch.float32), z(8, s), ts), (z(8, c // 4, dt=torch.int32), z(8, s), ts),
           (z(8, c), z(8, s, dt=torch.float32), ts), (z(8, c), z(8, s), torch.ones(1, dtype=torch.float64)),
           (z(8, c), z(8, s), torch.ones(1, dtype=torch.bfloat16))]
    for i, (codes, scales, scale) in enumerate(bad):
        W = mx.MXTensor(mx.FORMATS[fmt], 8, 64, codes, scales, scale)
        with pytest.raises(mx.MXError):
            mx._weights(W, -1)
        with pytest.raises(mx.MXError, match="expected|unsupported dtype"):
            mx.mx_linear(torch.zeros(4, 64, dtype=torch.bfloat16), W, torch.zeros(4, 8))


@pytest.mark.parametrize("fmt", SIZES)
def test_dense_bytes_of_the_size_are_taken(mx, fmt):
    c, s = SIZES[fmt]
    z = lambda *shape, dt=torch.uint8: torch.zeros(*shape, dtype=dt)
    ts = torch.ones(2) if fmt == "nvfp4" else None
    for codes, scales in ((z(8, c), z(8, s)), (z(8 * c), z(8 * s)), (z(16, c)[4:12], z(16, s)[4:12]),
                          (z(8, c).view(torch.int8), z(8, s).view(torch.float8_e4m3fn))):
        W = mx.MXTensor(mx.FORMATS[fmt], 8, 64, codes, scales, ts)
        assert mx._weights(W, -1) == bytes(W.desc())
    for rows, cols in ((0, 64), (8, 0)):
        W = mx.empty(mx.FORMATS[fmt], rows, cols, "cpu")
        assert mx._weights(W, -1) == bytes(W.desc())
