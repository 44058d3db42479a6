"""The example layer, forward and backward, against the layer in 64 bits with
the unquantized weights and the same choice of experts.

The bounds separate right wiring from wrong (which is off by 1 and more), not
rounding from rounding.  E2M1 steps are a third to a half of the value below
them, so a rounding moves an element by at most a fifth and by about a tenth
in the mean square; 8-bit checkpoints add 1/30.  A product of two NVFP4
matrices is then off by 0.15 of its norm, gate and up together by 0.25, the
second product by 0.3, and a gradient, which goes once more through a product,
by 0.35.  Twice that is allowed."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
    from moe_layer import MoELayer


def reference(layer, x, mask, d_out, d_loss):
    leaf = lambda t: t.detach().double().cpu().requires_grad_(True)
    x, router, w1, w2 = leaf(x), leaf(layer.router), leaf(layer.w1), leaf(layer.w2)
    r = layer.state["r"]
    chosen = r.experts.cpu().long()
    valid = mask.bool().cpu() if mask is not None else torch.ones(len(x), dtype=torch.bool)
    logits = x @ router.t()
    p = torch.softmax(logits, 1)
    out = torch.zeros_like(x)
    rows = []
    for t in range(len(x)):
        if not valid[t]:
            rows.append(torch.zeros_like(x[t]))
            continue
        w = torch.softmax(logits[t][chosen[t]], 0)
        acc = 0
        for j, e in enumerate(chosen[t].tolist()):
            h = w1[e] @ x[t]
            g, u = h.chunk(2)
            acc = acc + w[j] * (w2[e] @ (g * torch.sigmoid(g) * u))
        rows.append(acc)
    out = torch.stack(rows)
    counts = torch.bincount(chosen[valid].reshape(-1), minlength=layer.experts).double()
    V = valid.sum()
    loss = layer.experts / (layer.topk * V ** 2) * (counts * p[valid].sum(0)).sum()
    ((out * d_out.double().cpu()).sum() + d_loss * loss).backward()
    return out, loss, x.grad, router.grad, w1.grad, w2.grad


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk,padding",
                         [(65, 128, 64, 4, 2, False), (130, 96, 160, 6, 3, True), (1, 64, 32, 3, 1, False)])
def test_layer(tokens, hidden, inner, experts, topk, padding):
    layer = MoELayer(hidden, inner, experts, topk, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    d_out = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    mask = (torch.rand(tokens, generator=g, device="cuda") > 0.3).to(torch.uint8) if padding else None
    d_loss = torch.full((1,), 0.5, device="cuda")
    out, loss = layer.forward(x, mask)
    grads = layer.backward(d_out, d_loss)
    torch.cuda.synchronize()
    want = reference(layer, x, mask, d_out, 0.5)
    assert abs(loss.item() - want[1].item()) <= 1e-4 * want[1].item()
    for name, got, ref, bound in [("out", out, want[0], 0.6)] + [
            (n, a, b, 0.7) for n, a, b in zip(("dx", "router", "w1", "w2"), grads, want[2:])]:
        got = got.double().cpu()
        assert torch.isfinite(got).all(), name
        off = ((got - ref).norm() / ref.norm()).item() if ref.norm() > 0 else got.norm().item()
        print("%s off by %.3f of its norm" % (name, off))
        assert off <= bound, name
    if padding:
        assert bool((out[mask == 0] == 0).all())
