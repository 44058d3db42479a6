"""The sums of mx_logprob over long rows, where a lane adds many terms.

With U = 2^-24 the terms e^d of one value d carry one relative error: U |d| each for
the rounded factor scale / ln 2 and for the product, 2 U for the exponential.  Sums
of positive terms add U a rounding: 15 of 16 entries, 256 a run, one a run, 6 of
lanes and 8 of waves."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

U = 2.0 ** -24


@pytest.mark.parametrize("dtype,V", [("bf16", 2 ** 26), ("f32", 2 ** 25)])
def test_a_large_term_does_not_hide_the_small_ones(dtype, V):
    """One entry of weight 1 and V - 1 of e^-17.5, each less than half a step of it;
    65 rows with alternatives, so that a workgroup takes a row."""
    T = 65
    x = torch.full((T, V), -17.5, dtype={"bf16": torch.bfloat16, "f32": torch.float32}[dtype], device=dev())
    x[:, 5] = 0.0
    target = torch.full((T,), -1, device=dev())
    target[0], target[64] = 5, V - 1
    s = mx.mx_logprob(x, target, mx.logprobs(T, V, 1, dev()))
    rest = (V - 1) * math.exp(-17.5)
    share, ls = rest / (1 + rest), math.log1p(rest)
    runs = V / 512 / 16 / 256
    a = U * (15 + 256 + runs + 14 + share * (2 * 17.5 + 2))  # of the sum; of the other one, all terms of which are the small
    b = U * (15 + 256 + runs + 14 + 2 * 17.5 + 2 + 2)
    mean = 17.5 * share
    for t, at in ((0, 0.0), (64, -17.5)):
        assert abs(float(s.log_sum[t]) - ls) <= a + 2 * U * ls
        assert abs(float(s.logp[t]) - (at - ls)) <= a + 2 * U * ls + U * abs(at - ls)
        assert abs(float(s.entropy[t]) - (ls + mean)) <= a + 2 * U * ls + mean * (a + b + 3 * U) + U * (ls + mean)
        assert int(s.top_id[t, 0]) == 5
    d = mx.mx_logprob_backward(x, target, s, torch.ones(T, device=dev()), None, x)
    p = math.exp(-17.5 - ls)
    got = d[0, 6:4096].double()
    step = 2.0 ** -8 if dtype == "bf16" else U  # (the exponential 4 U, its argument's rounding 2 U (17.5 + ls))
    assert ((got + p).abs() <= p * (1.01 * step + a + U * (4 + 2 * (17.5 + ls)) + 2 * U * ls)).all()
    assert (d[1, ::65536] == 0).all()


@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** 100, 2.0 ** -100, 2.0 ** -149])
@pytest.mark.parametrize("V", [40, 100000])
def test_scales_at_the_ends(scale, V):
    """Far scales leave the largest entries alone or all entries alike: sums of 1s, which
    are exact, and a logarithm good to two steps."""
    x = torch.full((2, V), -3.0, device=dev())
    x[:, [4, V - 2]] = 1.0
    target = torch.tensor([4, 7], device=dev())
    s = mx.mx_logprob(x, target, mx.logprobs(2, V, 3, dev()), scale)
    n = 2 if scale > 1 else V
    assert (s.row_max == 1).all() and (s.log_sum.double() - math.log(n)).abs().max() <= 4 * U * math.log(n)
    assert (s.entropy.double() - math.log(n)).abs().max() <= 4 * U * math.log(n)
    assert float(s.logp[0]) == -float(s.log_sum[0]) and not torch.isnan(s.logp).any()
    assert s.top_id.tolist() == [[4, V - 2, 0]] * 2
    d = mx.mx_logprob_backward(x, target, s, torch.full((2,), min(1 / scale, 2.0 ** 100), device=dev()), None,
                               torch.empty_like(x), scale)
    assert torch.isfinite(d).all() and (d[0, 4] > 0).all() and (scale < 1 or (d[:, 9] == 0).all())
