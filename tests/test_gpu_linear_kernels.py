"""Each kernel of mx_linear on what does not change its results or changes them in
one place: pitched and shifted matrices, the residual in place, equal calls, another
stream, a graph, tokens and scales of NaN, nothing to sum.  Results are equal bits
throughout; test_gpu_more_operators.py checks the values."""
import pytest
import torch

from tests.linear_shapes import SHAPES

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMATS = ["mxfp4", "nvfp4", "mxfp8", "mxfp8_e5m2", "mxint8"]
K = 416  # three whole pairs of steps and a block behind them
SEED, COUNTER = 2 ** 50 + 7, 2 ** 32 - 3


def operands(fmt, M, N, K=K, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(N, K, generator=g, device=dev())
    amax = torch.zeros(1, device=dev()) if fmt == "nvfp4" else None
    W = mx.mx_quantize(w, mx.empty(mx.FORMATS[fmt], N, K, dev()), amax=amax)
    return torch.randn(M, K, generator=g, device=dev()).to(torch.bfloat16), W, g


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def pitched(like, pad, shift):
    """A matrix like `like` with a row pitch of `pad` more columns, `shift` elements into
    its allocation, and the allocation (of 99s)."""
    rows, cols = like.shape
    flat = torch.full((rows * (cols + pad) + shift + 8,), 99.0, dtype=like.dtype, device=dev())
    m = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(like)
    return m, flat


def gaps_stay(m, flat, pad, shift):
    rows, cols = m.shape
    end = shift + rows * (cols + pad)
    gap = flat[shift:end].view(rows, cols + pad)[:, cols:]
    return bool((gap == 99).all() and (flat[:shift] == 99).all() and (flat[end:] == 99).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kernel,number", [(k, i) for k in SHAPES for i in (0, 1)])
def test_pitch_and_alignment(kernel, number, dtype):
    M, N = SHAPES[kernel][number]
    x, W, g = operands("mxfp4", M, N)
    r = torch.randn(M, N, generator=g, device=dev()).to(TYPES[dtype])
    b = torch.randn(N, generator=g, device=dev())
    out, z = torch.empty_like(r), torch.empty_like(r)
    kw = dict(bias=b, act=mx.MX_ACT_GELU, drop=0.2, seed=SEED, counter=COUNTER)
    mx.mx_linear(x, W, out, z=z, residual=r, **kw)
    xp = pitched(x, 24, 8)[0]
    for pad, shift in ((8, 8), (3, 0), (5, 1)):
        (o2, fo), (z2, fz), (r2, fr) = (pitched(t, pad, shift) for t in (torch.zeros_like(r), torch.zeros_like(r), r))
        mx.mx_linear(xp, W, o2, z=z2, residual=r2, **kw)
        assert same(o2, out) and same(z2, z) and same(r2, r), (pad, shift)
        assert gaps_stay(o2, fo, pad, shift) and gaps_stay(z2, fz, pad, shift) and gaps_stay(r2, fr, pad, shift)
        mx.mx_linear(x, W, r2, residual=r2, **kw)  # in place, z not kept
        assert same(r2, out) and gaps_stay(r2, fr, pad, shift), (pad, shift)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel", SHAPES)
def test_equal_calls_streams_and_graphs(kernel, fmt):
    M, N = SHAPES[kernel][0]
    x, W, g = operands(fmt, M, N)
    r = torch.randn(M, N, generator=g, device=dev()).to(torch.bfloat16)
    kw = dict(act=mx.MX_ACT_SILU, residual=r, drop=0.1, seed=SEED, counter=COUNTER)
    first, second, side_out, graph_out = (torch.empty_like(r) for _ in range(4))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mx.mx_linear(x, W, side_out, stream=side, **kw)  # (two at once)
    mx.mx_linear(x, W, first, **kw)
    mx.mx_linear(x, W, second, **kw)
    torch.cuda.synchronize()
    assert same(first, second) and same(first, side_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_linear(x, W, graph_out, **kw)
    for i in range(3):
        x.copy_(torch.randn(M, K, generator=g, device=dev()))
        mx.mx_linear(x, W, first, **kw)
        graph_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(first, graph_out), i


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel", SHAPES)
def test_nan_and_infinity_stay_where_they_are(kernel, fmt):
    """Tokens of NaN or infinity change their rows alone, NaN scales their columns, in
    whole steps of K and in what is left of it."""
    M, N = SHAPES[kernel][0]
    x, W, g = operands(fmt, M, N)
    clean, out = torch.empty(M, N, device=dev()), torch.empty(M, N, device=dev())
    mx.mx_linear(x, W, clean)
    assert torch.isfinite(clean).all()
    nan = 0x7F if fmt == "nvfp4" else 255
    cols = torch.tensor(sorted({1, N // 2, N - 1}), device=dev())
    W.scales[cols[:-1], 0] = nan
    W.scales[cols[-1], -1] = nan
    mx.mx_linear(x, W, out)
    rest = torch.ones(N, dtype=torch.bool, device=dev())
    rest[cols] = False
    assert torch.isnan(out[:, cols]).all() and same(out[:, rest], clean[:, rest])
    x, W, g = operands(fmt, M, N)
    rows = torch.tensor(sorted({0, M // 2, M - 1}), device=dev())
    x[rows[0], K - 1] = float("nan")
    x[rows[1:], 5] = float("inf")
    mx.mx_linear(x, W, out)
    assert not torch.isfinite(out[rows][:, W.codes[:, 5 // (K // W.codes.shape[1])] & 0x70 != 0]).any()
    assert torch.isnan(out[rows[0]]).all()
    rest = torch.ones(M, dtype=torch.bool, device=dev())
    rest[rows] = False
    assert same(out[rest], clean[rest])


@pytest.mark.parametrize("kernel", SHAPES)
def test_nothing_to_sum(kernel):
    M, N = SHAPES[kernel][0]
    W = mx.empty(mx.FORMATS["mxfp8"], N, 0, dev())
    x = torch.empty(M, 0, dtype=torch.bfloat16, device=dev())
    b = torch.arange(N, device=dev()).float() - N / 2
    r, out, z = torch.ones(M, N, device=dev()), torch.full((M, N), 7.0, device=dev()), torch.empty(M, N, device=dev())
    mx.mx_linear(x, W, out, bias=b, act=mx.MX_ACT_RELU, residual=r, z=z)
    assert torch.equal(out, (b.clamp(min=0) + 1).expand(M, N)) and torch.equal(z, b.expand(M, N))


@pytest.mark.parametrize("kernel", SHAPES)
def test_every_block_scale_of_nvfp4(kernel):
    """One element of each column at each E4M3 scale, subnormal ones and the largest
    among them, times every code, against tokens of 1s: exact."""
    M, N = SHAPES[kernel][0]
    v = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    e4m3 = torch.arange(127, dtype=torch.uint8, device=dev())
    scales = e4m3.repeat(-(-N // 127))[:N]
    code = (torch.arange(N, device=dev()) // 127 * 3 + torch.arange(N, device=dev()) % 16) % 16
    values = torch.tensor(v + [-a for a in v], device=dev())[code]
    want = values * scales.view(torch.float8_e4m3fn).float()
    x = torch.ones(M, K, dtype=torch.bfloat16, device=dev())
    out = torch.empty(M, N, device=dev())
    for at in (3, 130, K - 1):  # (the last one in what is left of K)
        codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=dev())
        codes[:, at // 2] = (code << 4 * (at % 2)).to(torch.uint8)
        s = torch.zeros(N, K // 16, dtype=torch.uint8, device=dev())
        s[:, at // 16] = scales
        W = mx.MXTensor(mx.FORMATS["nvfp4"], N, K, codes, s, torch.full((1,), 0.25, device=dev()))
        mx.mx_linear(x, W, out)
        assert torch.equal(out, (want * 0.25).expand(M, N)), at
