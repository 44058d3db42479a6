"""Tensors whose offsets pass 32 bits, looked at in spots: the last rows and
the ones around 2^31 and 2^32."""
import pytest
import torch

pytestmark = [pytest.mark.gpu]

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev


def spots(rows, cols):
    at = {0, 1, rows - 2, rows - 1}
    for p in (31, 32, 33):
        r = (1 << p) // cols
        at |= {q for q in (r - 1, r, r + 1) if 0 <= q < rows}
    return torch.tensor(sorted(at), device=dev())


def fill(rows, cols, dtype=torch.bfloat16, seed=1):
    """Random values, a part at a time."""
    t = torch.empty(rows, cols, dtype=dtype, device=dev())
    g = torch.Generator(device="cuda").manual_seed(seed)
    for a in range(0, rows, 1 << 16):
        t[a:a + (1 << 16)].normal_(generator=g)
    return t


def test_swiglu():
    rows, cols = 530000, 4096  # 4.3e9 values of h
    h = fill(rows, 2 * cols)
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev())
    saved = mx.empty(mx.FORMATS["mxfp8"], rows, 2 * cols, dev())
    amax = torch.empty(1, device=dev())
    mx.mx_swiglu(h, y, saved=saved, amax=amax)
    at = spots(rows, 2 * cols)
    part = h[at].contiguous()
    y2, s2 = torch.empty(len(at), cols, dtype=torch.bfloat16, device=dev()), mx.empty(saved.fmt, len(at), 2 * cols, dev())
    mx.mx_swiglu(part, y2, saved=s2)
    assert torch.equal(y[at], y2) and torch.equal(saved.codes[at], s2.codes) and torch.equal(saved.scales[at], s2.scales)
    assert amax.item() == max(y[a:a + (1 << 16)].float().abs().max().item() for a in range(0, rows, 1 << 16))
    y8, y82 = mx.empty(saved.fmt, rows, cols, dev()), mx.empty(saved.fmt, len(at), cols, dev())
    dh2 = torch.empty_like(part)
    mx.mx_swiglu_backward(s2, y2, dh2, y_saved=y82)
    mx.mx_swiglu_backward(saved, y, h, y_saved=y8)
    assert torch.equal(h[at], dh2) and torch.equal(y8.codes[at], y82.codes) and torch.equal(y8.scales[at], y82.scales)


def test_combine():
    rows, cols, topk = 1100000, 4096, 2  # 4.5e9 values of Y
    Y = fill(rows, cols)
    at = spots(rows, cols)
    slots = torch.stack([at, at.flip(0)], 1).int().contiguous()
    w = torch.rand(len(at), topk, device=dev())
    out = torch.empty(len(at), cols, dtype=torch.bfloat16, device=dev())
    mx.mx_combine(Y, slots, w, out)
    want = (w[:, :, None] * Y[slots.long()].float()).sum(1)
    assert ((out.float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
    picked = Y[slots[:, 0].long()].float()
    dw = torch.empty_like(w)
    single = slots[:, :1].contiguous()
    dY = torch.zeros_like(Y)
    mx.mx_combine_backward(out, Y, single, w[:, :1].contiguous(), dY, dw[:, :1].contiguous())
    want = w[:, :1] * out.float()
    assert ((dY[at].float() - want).abs() <= 2.0 ** -8 * want.abs()).all()
    dw = torch.empty(len(at), 1, device=dev())
    mx.mx_combine_backward(out, Y, single, None, None, dw)
    prod = out.double() * picked.double()
    assert ((dw[:, 0].double() - prod.sum(1)).abs() <= cols * 2.0 ** -23 * prod.abs().sum(1)).all()


def test_wgrad():
    x_rows, K, N, R = 600000, 7232, 64, 512  # 4.3e9 codes of X
    X = mx.empty(mx.FORMATS["mxint8"], x_rows, K, dev())
    g = torch.Generator(device="cuda").manual_seed(2)
    for a in range(0, x_rows, 1 << 16):
        X.codes[a:a + (1 << 16)].random_(0, 256, generator=g)
    X.scales.random_(120, 130, generator=g)
    at = spots(x_rows, K)
    index = at[torch.randint(0, len(at), (R,), generator=g, device=dev())].int().contiguous()
    dy = torch.randn(R, N, generator=g, device=dev()).to(torch.bfloat16)
    off = torch.tensor([0, 200, R], dtype=torch.int64, device=dev())
    dw = torch.empty(2 * N, K, device=dev())
    mx.mx_wgrad_grouped(dy, X, index, 2, off, dw)
    few = mx.MXTensor(X.fmt, len(at), K, X.codes[at].contiguous(), X.scales[at].contiguous())
    x = torch.empty(len(at), K, device=dev())
    mx.mx_dequantize(few, x)
    x = x[torch.searchsorted(at, index.long())].double()
    for e, (a, b) in enumerate(((0, 200), (200, R))):
        d = dy[a:b].double()
        want, mag = d.t() @ x[a:b], d.abs().t() @ x[a:b].abs()
        assert ((dw[e * N:(e + 1) * N].double() - want).abs() <= (b - a + 2) * 2.0 ** -23 * mag).all()


def test_wgrad_of_a_large_gradient():
    E, N, K, R = 70, 4096, 8192, 300  # 2.3e9 values of dW
    X = mx.empty(mx.FORMATS["mxfp8"], R, K, dev())
    mx.mx_quantize(torch.randn(R, K, device=dev()), X)
    x = torch.empty(R, K, device=dev())
    mx.mx_dequantize(X, x)
    dy = torch.randn(R, N, device=dev()).to(torch.bfloat16)
    off = torch.tensor([0] * 64 + [100, 100, 100, 100, 250, 250, R], dtype=torch.int64, device=dev())
    dw = torch.full((E * N, K), 7.0, device=dev())
    mx.mx_wgrad_grouped(dy, X, None, E, off, dw)
    for e in (0, 62, 63, 64, 67, 68, 69):
        a, b = int(off[e]), int(off[e + 1])
        want, mag = dy[a:b].double().t() @ x[a:b].double(), dy[a:b].double().abs().t() @ x[a:b].double().abs()
        assert ((dw[e * N:(e + 1) * N].double() - want).abs() <= (b - a + 2) * 2.0 ** -23 * mag).all(), e


def test_route():
    tokens, experts, topk = mx.MX_ROUTE_MAX_TOKENS, 520, 1  # 4.4e9 scores
    logits = fill(tokens, experts, seed=3)
    r = mx.routing(tokens, experts, topk, dev())
    mx.mx_route(logits, r)
    at = spots(tokens, experts)
    small = mx.routing(len(at), experts, topk, dev())
    part = logits[at].contiguous()
    mx.mx_route(part, small)
    assert torch.equal(r.experts[at], small.experts) and torch.equal(r.weights[at], small.weights)
    assert torch.equal(r.counts, torch.bincount(r.experts.view(-1), minlength=experts))
    assert torch.equal(r.group_offsets[1:], r.counts.cumsum(0)) and r.group_offsets[0] == 0
    slot = r.slot_row.view(-1).long()
    assert torch.equal(r.row_index[slot], torch.arange(tokens, dtype=torch.int32, device=dev()))
    assert torch.equal(torch.searchsorted(r.group_offsets, slot, right=True) - 1, r.experts.view(-1).long())
    dw = torch.rand(tokens, topk, device=dev())
    d = torch.empty(len(at), experts, dtype=torch.bfloat16, device=dev())
    mx.mx_route_backward(part, small, dw[at].contiguous(), None, d)
    whole = torch.empty_like(logits)
    mx.mx_route_backward(logits, r, dw, None, whole)
    assert torch.equal(whole[at], d)
