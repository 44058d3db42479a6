"""A feed-forward block and a scoring head out of the library's calls, forward and
backward, as a policy gradient uses them.

    y = x + drop(W2 gelu(W1 x + b1) + b2),   logits = H y,
    log probabilities of the given tokens and entropies of the rows

Weights are kept in a block-scaled 8-bit format (and once more transposed, for the
gradients of the activations), activations in bf16; what the weights' gradients need
of the activations is kept in 8 bits.  Run on a GPU:  python examples/dense_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import microscaling_precision_gemm_amd as mx  # noqa: E402

SAVED = mx.FORMATS["mxfp8"]


def quantized(w, fmt):
    return mx.mx_quantize(w.contiguous(), mx.empty(fmt, *w.shape, device=w.device))


class ScoredBlock:
    def __init__(self, hidden, inner, vocab, drop=0.1, weights="mxfp8", saved=SAVED, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g, device=device) / s[-1] ** 0.5
        self.hidden, self.inner, self.vocab, self.drop = hidden, inner, vocab, drop
        self.fmt, self.saved, self.seed, self.counter = mx.FORMATS[weights], saved, seed + 1, 0
        self.w1, self.w2, self.head = new(inner, hidden), new(hidden, inner), new(vocab, hidden)
        self.b1, self.b2 = new(inner) * 0.1, new(hidden) * 0.1
        self.quantize_weights()

    def quantize_weights(self):
        """After every change of the weights."""
        self.q = {n: quantized(getattr(self, n), self.fmt) for n in ("w1", "w2", "head")}
        self.qt = {n: quantized(getattr(self, n).t(), self.fmt) for n in ("w1", "w2", "head")}

    def eight_bit(self, x):
        return mx.mx_quantize(x, mx.empty(self.saved, *x.shape, device=x.device))

    def forward(self, x, target, topk=0):
        """x [tokens, hidden] bf16, target int64 [tokens] (-1: padding) -> the scoring (mx.Logprobs)."""
        T, dev = len(x), x.device
        new = lambda n: torch.empty(T, n, dtype=torch.bfloat16, device=dev)
        s = self.state = {"target": target, "counter": self.counter}
        self.counter += T * -(-self.hidden // 8)  # the next call draws other masks
        s["z"], h, y, s["logits"] = new(self.inner), new(self.inner), new(self.hidden), new(self.vocab)
        mx.mx_linear(x, self.q["w1"], h, bias=self.b1, act=mx.MX_ACT_GELU, z=s["z"])
        mx.mx_linear(h, self.q["w2"], y, bias=self.b2, residual=x, drop=self.drop, seed=self.seed,
                     counter=s["counter"])
        mx.mx_linear(y, self.q["head"], s["logits"])
        s["x8"], s["h8"], s["y8"] = self.eight_bit(x), self.eight_bit(h), self.eight_bit(y)
        s["scores"] = mx.mx_logprob(s["logits"], target, mx.logprobs(T, self.vocab, topk, dev))
        return s["scores"]

    def backward(self, d_logp, d_entropy):
        """Gradients (x in bf16, the weights' and biases' in fp32)."""
        s, T, dev = self.state, len(d_logp), d_logp.device
        new = lambda n: torch.empty(T, n, dtype=torch.bfloat16, device=dev)

        def weight(d, x8):
            d_w = torch.empty(d.shape[1], x8.cols, device=dev)
            return mx.mx_wgrad_grouped(d, x8, None, 1, None, d_w)

        # (the logits are not needed any more)
        d_logits = mx.mx_logprob_backward(s["logits"], s["target"], s["scores"], d_logp, d_entropy, s["logits"])
        d_head = weight(d_logits, s["y8"])
        d_y = mx.mx_linear(d_logits, self.qt["head"], new(self.hidden))
        d_b1, d_b2 = torch.empty_like(self.b1), torch.empty_like(self.b2)
        d_z2, _ = mx.mx_epilogue_backward(d_y, None, new(self.hidden), d_b2, drop=self.drop, seed=self.seed,
                                          counter=s["counter"])
        d_w2 = weight(d_z2, s["h8"])
        d_h = mx.mx_linear(d_z2, self.qt["w2"], new(self.inner))
        d_z1, _ = mx.mx_epilogue_backward(d_h, s["z"], d_h, d_b1, act=mx.MX_ACT_GELU)
        d_w1 = weight(d_z1, s["x8"])
        d_x = mx.mx_linear(d_z1, self.qt["w1"], new(self.hidden), residual=d_y)
        return {"x": d_x, "w1": d_w1, "b1": d_b1, "w2": d_w2, "b2": d_b2, "head": d_head}


def main(tokens=4096, hidden=4096, inner=14336, vocab=32000, steps=5):
    block = ScoredBlock(hidden, inner, vocab)
    x = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    target = torch.randint(0, vocab, (tokens,), device="cuda")
    d_logp = torch.randn(tokens, device="cuda") / tokens
    d_entropy = torch.full((tokens,), -0.01 / tokens, device="cuda")
    for i in range(steps):
        a, b, c = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        a.record()
        scores = block.forward(x, target)
        b.record()
        block.backward(d_logp, d_entropy)
        c.record()
        torch.cuda.synchronize()
        print("step %d: forward %.3f ms, backward %.3f ms, mean log probability %.4f" %
              (i, a.elapsed_time(b), b.elapsed_time(c), scores.logp.mean().item()), flush=True)


if __name__ == "__main__":
    main()
