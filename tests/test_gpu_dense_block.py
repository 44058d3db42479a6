"""The example block, forward and backward, against the block in 64 bits with the
unquantized weights and the same dropout mask; and the calls recorded into a graph.

The bounds separate right wiring from wrong (which is off by 1 and more), not
rounding from rounding.  With 8-bit integers a weight is off by 2^-6 / sqrt 12 of its
block's power of two, which is at most the largest of 32 normal values, about 2.2
deviations: 0.010 of the weights' norm; bf16 activations add 0.003 a product.  A
gradient goes through the scores (whose logits, of size 1, are off by 0.02) and up to
five such products: 0.05.  Twice that is allowed."""
import os
import sys

import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
    import microscaling_precision_gemm_amd as mx
    from dense_block import ScoredBlock
    from tests.gpu_util import dev


def reference(block, x, target, counter, d_logp, d_entropy):
    leaf = lambda t: t.detach().double().cpu().requires_grad_(True)
    p = {n: leaf(getattr(block, n)) for n in ("w1", "b1", "w2", "b2", "head")}
    p["x"] = leaf(x)
    mask = torch.from_numpy(R.drop_factors(block.drop, block.seed, counter, len(x), block.hidden))
    z = p["x"] @ p["w1"].t() + p["b1"]
    h = 0.5 * z * torch.special.erfc(-z / 2 ** 0.5)
    y = p["x"] + (h @ p["w2"].t() + p["b2"]) * mask
    q = torch.log_softmax(y @ p["head"].t(), 1)
    there = (target >= 0).cpu()
    logp = torch.where(there, q.gather(1, target.clamp(min=0).cpu()[:, None])[:, 0], 0.0)
    entropy = torch.where(there, -(q.exp() * q).sum(1), 0.0)
    (d_logp.double().cpu() * logp + d_entropy.double().cpu() * entropy).sum().backward()
    return logp.detach(), entropy.detach(), {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("tokens,hidden,inner,vocab", [(96, 128, 256, 512), (300, 256, 160, 1056), (7, 64, 96, 320)])
def test_block(tokens, hidden, inner, vocab):
    block = ScoredBlock(hidden, inner, vocab, drop=0.25, weights="mxint8", saved=mx.FORMATS["mxint8"], seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    for step in range(2):  # the second step draws another mask
        x = torch.randn(tokens, hidden, generator=g, device=dev()).to(torch.bfloat16)
        target = torch.randint(-1, vocab, (tokens,), generator=g, device=dev())
        d_logp, d_entropy = (torch.randn(tokens, generator=g, device=dev()) for _ in range(2))
        counter = block.counter
        scores = block.forward(x, target, topk=3)
        grads = block.backward(d_logp, d_entropy)
        logp, entropy, want = reference(block, x, target, counter, d_logp, d_entropy)
        assert (scores.logp.double().cpu() - logp).abs().max() < 0.1
        assert (scores.entropy.double().cpu() - entropy).abs().max() < 0.1
        for n, w in want.items():
            err = (grads[n].double().cpu() - w).norm() / w.norm()
            assert err < 0.1, (step, n, float(err))


@pytest.mark.parametrize("tokens", [1, 40, 200])
def test_replays_equal_direct_calls(tokens):
    hidden, inner, vocab = 128, 288, 5000
    block = ScoredBlock(hidden, inner, vocab - vocab % 32, weights="mxfp4")
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g, device=dev()).to(torch.bfloat16)
    target = torch.randint(0, block.vocab, (tokens,), generator=g, device=dev())
    new = lambda n, dt=torch.bfloat16: torch.empty(tokens, n, dtype=dt, device=dev())
    z, h, y, logits = new(inner), new(inner), new(hidden), new(block.vocab)
    d_logits, d_z, d_bias = new(block.vocab), new(inner), torch.empty(inner, device=dev())
    d_logp = torch.randn(tokens, generator=g, device=dev())
    s = mx.logprobs(tokens, block.vocab, 5, dev())
    ws = torch.empty(mx.mx_epilogue_workspace_bytes(tokens, inner), dtype=torch.uint8, device=dev())
    dropped = new(hidden)
    state = [z, h, y, logits, d_logits, d_z, d_bias, dropped, s.logp, s.entropy, s.row_max, s.log_sum, s.top_id,
             s.top_logp]

    def step():
        mx.mx_linear(x, block.q["w1"], h, bias=block.b1, act=mx.MX_ACT_SILU, z=z)
        mx.mx_linear(h, block.q["w2"], y, bias=block.b2, residual=x, drop=0.1, seed=3, counter=9)
        mx.mx_dropout(y, dropped, 0.5, 3, 10 ** 6)
        mx.mx_linear(y, block.q["head"], logits)
        mx.mx_logprob(logits, target, s)
        mx.mx_logprob_backward(logits, target, s, d_logp, None, d_logits)
        mx.mx_epilogue_backward(h, z, d_z, d_bias, act=mx.MX_ACT_SILU, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(tokens, hidden, generator=g, device=dev()))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in state]
        for t in state:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(state, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, n)
        ws.fill_(i + 1)
