"""The scales that token scoring takes: those whose quotient by ln 2 is an FP32 number."""
import ctypes

import pytest

from tests.test_abi_dense import ALIGN, FAKE, UNSUP, mx, scoring  # noqa: F401


@pytest.mark.parametrize("scale,ok", [(2.0 ** 127, True), (1e-45, True), (1.0, True), (2.0 ** 127 * (1 + 2.0 ** -23), False),
                                      (2.4e38, False), (3.4e38, False)])
def test_scale(mx, scale, ok):  # noqa: F811
    L, p = mx.load(), scoring(mx)
    # an accepted scale gets as far as the misaligned logits
    want = ALIGN if ok else UNSUP
    f = ctypes.c_float(scale)
    assert L.mx_logprob(FAKE + 1, 0, 50, FAKE, f, p, None, 0, None) == want
    assert L.mx_logprob_backward(FAKE + 1, 0, 50, FAKE, f, p, FAKE, FAKE, FAKE, 50, None) == want
