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


@pytest.mark.parametrize("T,E,topk,kind,normalize", [(16385, 256, 8, "f32", True), (40003, 60, 4, "bf16", True),
                                                     (40003, 24, 3, "f32", False), (5001, 300, 2, "f32", True)])
def test_a_group_of_lanes_does_several_tokens(T, E, topk, kind, normalize):
    """More tokens than the grid has groups of lanes (16384 of 16 lanes up to 256
    experts, 4096 above): a later token gets the bits it gets alone, whatever
    came before it, padding and rows without a choice among them."""
    mask = np.random.default_rng(3).random(T) > 0.2
    x, r, m, dw = routed(T, E, topk, kind, 3, normalize, mask=mask, holes=0.1)
    x[5::97] = -float("inf")
    r = mx.mx_route(x, r, token_mask=m, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    dl = torch.tensor([30.0], device=dev())
    d = backward(x, r, m, dw, dl, normalize)
    assert not bool(d[~torch.from_numpy(mask).to(dev())].any())
    for a in range(0, T, 4001):
        n = min(4001, T - a)
        part = mx.routing(n, E, topk, device=dev())
        for name in ("experts", "counts", "valid"):  # the whole batch's counts: the loss is the batch's
            whole = getattr(r, name)
            getattr(part, name).copy_(whole[a:a + n] if name == "experts" else whole)
        got = backward(x[a:a + n].contiguous(), part, m[a:a + n].contiguous(), dw[a:a + n].contiguous(), dl, normalize)
        assert torch.equal(d[a:a + n], got), a
    p = torch.softmax(x.double(), 1).nan_to_num(0.0) * torch.from_numpy(mask).to(dev())[:, None]
    there = r.experts >= 0
    at = r.experts.long().clamp(min=0)
    b = 30.0 * E / (topk * float(r.valid) ** 2) * r.counts.double()
    w = torch.where(there, dw, 0.0).double()
    q = torch.zeros_like(p).scatter_add_(1, at, torch.where(there, p.gather(1, at), 0.0))
    if normalize:
        q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
    hot = torch.zeros_like(p).scatter_add_(1, at, w)
    pb, pa, qd, qa = ((v * c).sum(1, keepdim=True) for v, c in ((p, b), (p, b.abs()), (q, hot), (q, hot.abs())))
    other = q if normalize else p
    want = p * (b - pb) + q * hot - other * qd
    size = p * (b.abs() + pa) + q * hot.abs() + other * qa
    # p and q to 29 * 2^-24, differences of scores 2^-24 of up to 10, sums and roundings 40 more
    tol = 128 * 2.0 ** -24 * size + 1e-37 + (2.0 ** -8 * want.abs() if kind == "bf16" else 0)
    assert bool(((d.double() - want).abs() <= tol).all())
