"""The router's gradient where something is not there: slots without an expert
and padding tokens."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def routed(T, E, topk, kind, seed, normalize, mask=None, holes=0.0):
    """Scores (a part of them -inf), their routing, and random gradients of the weights."""
    g = np.random.default_rng([seed, T, E])
    x = g.standard_normal((T, E)).astype(np.float32)
    x[g.random((T, E)) < holes] = -np.inf
    x = torch.from_numpy(x).to(dev()).to(DT[kind])
    m = None if mask is None else torch.from_numpy(mask.astype(np.uint8)).to(dev())
    r = mx.routing(T, E, topk, device=dev())
    mx.mx_route(x, r, token_mask=m, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    dw = torch.from_numpy(g.standard_normal((T, topk)).astype(np.float32)).to(dev())
    return x, r, m, dw


def backward(x, r, m, dw, dl, normalize):
    d = torch.full_like(x, 7.0)
    mx.mx_route_backward(x, r, dw, dl, d, token_mask=m, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    torch.cuda.synchronize()
    return d


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,topk", [(40, 6, 5), (33, 30, 16), (20, 300, 4)])
def test_gradients_of_empty_slots_are_not_looked_at(T, E, topk, kind, normalize):
    """An empty slot's weight is 0 whatever the scores are, so what its gradient
    holds (it may never have been written) changes nothing."""
    x, r, m, dw = routed(T, E, topk, kind, 1, normalize, holes=1 - topk / E / 2)
    empty = r.experts < 0
    assert bool(empty.any()) and not bool(empty.all())
    dl = torch.tensor([0.5], device=dev())
    want = backward(x, r, m, torch.where(empty, 0.0, dw), dl, normalize)
    assert bool(torch.isfinite(want).all())
    for junk in (float("nan"), float("inf"), -float("inf"), 3e38):
        assert torch.equal(backward(x, r, m, torch.where(empty, junk, dw), dl, normalize), want), junk


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,topk", [(40, 6, 2), (65, 40, 8), (20, 300, 4)])
def test_padding_gets_zeros_whatever_the_loss(T, E, topk, kind, normalize):
    """A loss that overflowed shows in the tokens, not in the padding."""
    mask = np.arange(T) % 3 != 1
    x, r, m, dw = routed(T, E, topk, kind, 2, normalize, mask=mask)
    x[1] = float("nan")
    for bad in (float("nan"), float("inf"), -float("inf")):
        d = backward(x, r, m, dw, torch.tensor([bad], device=dev()), normalize)
        assert not bool(d[~torch.from_numpy(mask).to(dev())].any()), bad
        assert not bool(torch.isfinite(d[torch.from_numpy(mask).to(dev())]).any()), bad
