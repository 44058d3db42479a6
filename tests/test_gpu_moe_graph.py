"""The router, activation, weight gradient and combination recorded into one
graph: every replay equals the direct calls, with other work between them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev


@pytest.mark.parametrize("tokens,experts,topk,cols", [(1, 8, 2, 64), (700, 40, 4, 160), (5000, 16, 2, 96)])
def test_replays_equal_direct_calls(tokens, experts, topk, cols):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    new = lambda *s: torch.randn(*s, generator=g, device=dev())
    rows = tokens * topk
    logits, h = new(tokens, experts), new(rows, 2 * cols).to(torch.bfloat16)
    d_out, d_loss = new(tokens, cols).to(torch.bfloat16), new(1)
    saved, y8 = mx.empty(mx.FORMATS["mxfp8"], rows, 2 * cols, dev()), mx.empty(mx.FORMATS["mxint8"], rows, cols, dev())
    r = mx.routing(tokens, experts, topk, dev())
    o = dict(y=torch.empty(rows, cols, dtype=torch.bfloat16, device=dev()), amax=torch.empty(1, device=dev()),
             out=torch.empty_like(d_out), dz=torch.empty(rows, cols, dtype=torch.bfloat16, device=dev()),
             dw=torch.empty(tokens, topk, device=dev()), dh=torch.empty_like(h),
             dx=torch.empty_like(logits), dW=torch.empty(experts * cols, cols, device=dev()))
    ws = torch.empty(mx.mx_wgrad_workspace_bytes(rows, cols, cols, experts), dtype=torch.uint8, device=dev())
    state = [r.experts, r.weights, r.slot_row, r.row_index, r.group_offsets, r.counts, r.valid, r.prob_sum, r.loss,
             saved.codes, saved.scales, y8.codes, y8.scales] + list(o.values())

    def step():
        mx.mx_route(logits, r)
        mx.mx_swiglu(h, o["y"], saved=saved, amax=o["amax"])
        mx.mx_combine(o["y"], r.slot_row, r.weights, o["out"])
        mx.mx_combine_backward(d_out, o["y"], r.slot_row, r.weights, o["dz"], o["dw"])
        mx.mx_swiglu_backward(saved, o["dz"], o["dh"], y_saved=y8)
        mx.mx_wgrad_grouped(o["dz"], y8, None, experts, r.group_offsets, o["dW"], workspace=ws)
        mx.mx_route_backward(logits, r, o["dw"], d_loss, o["dx"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        h.copy_(new(rows, 2 * cols))
        logits.copy_(new(tokens, experts))
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
