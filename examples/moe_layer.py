"""A mixture-of-experts layer out of the library's calls, forward and backward.

    out[t] = sum over the token's chosen experts e of weight * W2_e swiglu(W1_e x[t])

Expert products run in NVFP4 (mx_gemm_grouped); what the backward pass needs of
the activations is kept in 8 bits (MXFP8): the tokens, and the inputs of the
gated activation.  Sizes: tokens x hidden, experts of `inner` columns, topk a
token.  Run on a GPU:  python examples/moe_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import microscaling_precision_gemm_amd as mx  # noqa: E402

SAVED = mx.FORMATS["mxfp8"]
NVFP4 = mx.FORMATS["nvfp4"]


def nvfp4(x, amax=None):
    """x in NVFP4; amax: its largest magnitude, if known."""
    q = mx.empty(NVFP4, *x.shape, device=x.device)
    if amax is not None:
        return mx.mx_quantize(x, q, flags=mx.MX_FLAG_AMAX_GIVEN, amax=amax)
    return mx.mx_quantize(x, q, amax=torch.empty(1, dtype=torch.float32, device=x.device))


def nvfp4_experts(w):
    """The stacked experts [E, N, K] in NVFP4, a tensor scale for each."""
    E, N, K = w.shape
    q = mx.empty(NVFP4, E * N, K, device=w.device, n_tensor_scales=E)
    amax = torch.empty(E, dtype=torch.float32, device=w.device)
    mx.mx_quantize_batch([dict(x=w[e], out=q.view_rows(e * N, (e + 1) * N, q.tensor_scale[e:e + 1]),
                               amax=amax[e:e + 1]) for e in range(E)])
    return q


class MoELayer:
    def __init__(self, hidden, inner, experts, topk, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g, device=device) / s[-1] ** 0.5
        self.hidden, self.inner, self.experts, self.topk = hidden, inner, experts, topk
        self.router = new(experts, hidden)
        self.w1 = new(experts, 2 * inner, hidden)  # gate rows, then up rows
        self.w2 = new(experts, hidden, inner)
        self.quantize_weights()

    def quantize_weights(self):
        """After every change of the weights."""
        self.q1, self.q2 = nvfp4_experts(self.w1), nvfp4_experts(self.w2)
        self.q1t = nvfp4_experts(self.w1.transpose(1, 2).contiguous())
        self.q2t = nvfp4_experts(self.w2.transpose(1, 2).contiguous())

    def product(self, q, rows, weights, r, width, row_index=None):
        # (rows past the last group, of tokens without a choice, stay 0)
        out = torch.zeros(rows, width, dtype=torch.bfloat16, device=q.codes.device)
        return mx.mx_gemm_grouped(q, row_index, rows, weights, self.experts, r.group_offsets, out)

    def forward(self, x, token_mask=None):
        """x [tokens, hidden] bf16 -> (out, balance loss)."""
        T, R = x.shape[0], x.shape[0] * self.topk
        s = self.state = {"mask": token_mask}
        s["x"], s["logits"] = x, x.float() @ self.router.t()
        r = s["r"] = mx.routing(T, self.experts, self.topk, x.device)
        mx.mx_route(s["logits"], r, token_mask, flags=mx.MX_ROUTE_NORMALIZE)
        s["x8"] = mx.mx_quantize(x, mx.empty(SAVED, T, self.hidden, x.device))
        h = self.product(nvfp4(x), R, self.q1, r, 2 * self.inner, r.row_index)
        y = torch.empty(R, self.inner, dtype=torch.bfloat16, device=x.device)
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
        s["h8"] = mx.empty(SAVED, R, 2 * self.inner, x.device)
        mx.mx_swiglu(h, y, saved=s["h8"], amax=amax)
        s["z"] = self.product(nvfp4(y, amax), R, self.q2, r, self.hidden)
        return mx.mx_combine(s["z"], r.slot_row, r.weights, torch.empty_like(x)), r.loss

    def backward(self, d_out, d_loss=None):
        """Gradients of x, router, w1, w2 (fp32, x in bf16)."""
        s, r = self.state, self.state["r"]
        R, dev = s["z"].shape[0], d_out.device
        E, H, F = self.experts, self.hidden, self.inner
        dz, dw = torch.zeros_like(s["z"]), torch.empty_like(r.weights)
        mx.mx_combine_backward(d_out, s["z"], r.slot_row, r.weights, dz, dw)
        dy = self.product(nvfp4(dz), R, self.q2t, r, F)
        dh = torch.empty(R, 2 * F, dtype=torch.bfloat16, device=dev)
        y8 = mx.empty(SAVED, R, F, dev)
        mx.mx_swiglu_backward(s["h8"], dy, dh, y_saved=y8)
        d_w2 = torch.empty(E * H, F, device=dev)
        mx.mx_wgrad_grouped(dz, y8, None, E, r.group_offsets, d_w2)
        d_w1 = torch.empty(E * 2 * F, H, device=dev)
        mx.mx_wgrad_grouped(dh, s["x8"], r.row_index, E, r.group_offsets, d_w1)
        dx_rows = self.product(nvfp4(dh), R, self.q1t, r, H)
        dx = mx.mx_combine(dx_rows, r.slot_row, None, torch.empty_like(d_out))
        d_logits = torch.empty_like(s["logits"])
        mx.mx_route_backward(s["logits"], r, dw, d_loss, d_logits, s["mask"], flags=mx.MX_ROUTE_NORMALIZE)
        dx = (dx.float() + d_logits @ self.router).to(dx.dtype)
        return dx, d_logits.t() @ s["x"].float(), d_w1.view_as(self.w1), d_w2.view_as(self.w2)


def main(tokens=4096, hidden=2048, inner=1024, experts=32, topk=8, steps=5):
    layer = MoELayer(hidden, inner, experts, topk)
    x = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    d_out = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    d_loss = torch.full((1,), 0.01, device="cuda")
    for i in range(steps):
        a, b, c = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        a.record()
        out, loss = layer.forward(x)
        b.record()
        layer.backward(d_out, d_loss)
        c.record()
        torch.cuda.synchronize()
        print("step %d: forward %.3f ms, backward %.3f ms, balance loss %.4f" %
              (i, a.elapsed_time(b), b.elapsed_time(c), loss.item()), flush=True)


if __name__ == "__main__":
    main()
