"""mx_linear against its formula in 64 bits: every weight format, epilogue and kind
of size, strides and alignments, extreme weights, equal calls."""
import numpy as np
import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMATS = ["mxfp4", "nvfp4", "mxfp8", "mxfp8_e5m2", "mxint8"]


def random_weights(g, fmt, n, k):
    """Codes of every kind but NaN and infinity, scales over a few octaves."""
    four = fmt in ("mxfp4", "nvfp4")
    codes = g.integers(0, 256, (n, k // 2 if four else k), dtype=np.uint8)
    if not four:
        codes = np.where(np.isnan(R.eight_bit_values(fmt)[codes]), np.uint8(7), codes)
    if fmt == "nvfp4":
        return codes, g.integers(40, 96, (n, k // 16), dtype=np.uint8), np.float32(g.uniform(0.01, 0.02))
    if fmt == "mxfp8_e5m2":  # (its elements alone span 30 octaves)
        codes = codes & 0xBF | np.uint8(0x20)
    return codes, g.integers(118, 124, (n, k // 32), dtype=np.uint8), None


def upload(fmt, codes, scales, ts):
    n, k = len(codes), scales.shape[1] * (16 if fmt == "nvfp4" else 32)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    return mx.MXTensor(mx.FORMATS[fmt], n, k, to(codes), to(scales),
                       None if ts is None else torch.tensor([ts], device=dev()))


def matrix(values, dtype, pad=0, shift=0):
    """values on the device with a row pitch of `pad` more columns, starting
    `shift` elements into its allocation; and what it holds, in 64 bits"""
    rows, cols = values.shape
    flat = torch.full((rows * (cols + pad) + shift + 8,), 99.0, dtype=TYPES[dtype], device=dev())
    m = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.from_numpy(values))
    return m, m.double().cpu().numpy()


def check(got, want, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), [(tuple(i), got[tuple(i)], want[tuple(i)], tol[tuple(i)])
                                                  for i in np.argwhere(bad)[:4]])


def run(seed, M, N, K, fmt, dtype="bf16", bias=None, act="none", drop=0.0, residual=False, keep_z=False, pad=0,
        shift=0, in_place=False):
    g = np.random.default_rng(seed)
    codes, scales, ts = random_weights(g, fmt, N, K)
    W = upload(fmt, codes, scales, ts)
    w = R.weights(fmt, codes, scales, 1.0 if ts is None else ts)
    x, x64 = matrix(g.normal(size=(M, K)), "bf16", pad=8 * (pad > 0))
    size = max(np.sqrt(K) * 0.25, 1.0)
    b = b64 = r = r64 = z = None
    if bias:
        b = torch.from_numpy(g.normal(size=N) * size).to(TYPES[bias]).to(dev())
        b64 = b.double().cpu().numpy()
    if residual or in_place:
        r, r64 = matrix(g.normal(size=(M, N)) * size, dtype, pad, shift)
    out = r if in_place else matrix(np.zeros((M, N)), dtype, pad, shift)[0]
    if keep_z:
        z, _ = matrix(np.zeros((M, N)), dtype, pad, shift)
    seed_, counter = 2 ** 50 + seed, 2 ** 32 - 5
    mx.mx_linear(x, W, out, bias=b, act=mx.ACTIVATIONS[act], z=z, residual=r, drop=drop, seed=seed_, counter=counter)
    torch.cuda.synchronize()
    fac = R.drop_factors(drop, seed_, counter, M, N) if drop else None
    (zw, zt), (ow, ot) = R.linear(x64, w, b64, act, fac, r64, dtype)
    if keep_z:
        check(z, zw, zt, "z")
    check(out, ow, ot, "out")
    if pad and out.storage_offset() == shift:  # what lies between the rows stays
        gap = out.as_strided((M, pad), (N + pad, 1), shift + N)
        assert (gap == 99).all()
    return x, W, b, r, out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 130, 288), (2, 17, 64), (3, 4099, 96), (16, 64, 1024), (17, 33, 160),
                                   (31, 256, 352), (33, 72, 544), (64, 200, 256), (65, 129, 2080), (130, 256, 512),
                                   (300, 520, 384)])
def test_formats_and_sizes(fmt, M, N, K):
    run(M + N, M, N, K, fmt, bias="f32", act="gelu")


@pytest.mark.parametrize("M,N,K", [(256, 256, 128), (257, 513, 256), (512, 1024, 640), (1000, 776, 1152),
                                   (2048, 512, 384)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_batches(fmt, M, N, K):
    run(M * 3 + N, M, N, K, fmt, bias="bf16", act="silu", residual=True, drop=0.1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(70, 130, 32), (100, 264, 64), (20, 96, 96), (90, 200, 224), (300, 264, 1056),
                                   (1030, 1300, 96), (1500, 1000, 288), (1900, 1040, 192)])
def test_ragged_sums(fmt, M, N, K):
    run(M + K, M, N, K, fmt, bias="f32", act="gelu_tanh", keep_z=True)


@pytest.mark.parametrize("fmt,K", [("mxfp4", 128), ("nvfp4", 160), ("mxfp8", 192), ("mxfp8_e5m2", 224),
                                   ("mxint8", 256), ("mxfp4", 32), ("nvfp4", 384), ("mxfp8", 640)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_tiles(fmt, K, dtype):
    """A whole round of the largest tiles, the last ones not full."""
    run(K, 2040, 8190, K, fmt, dtype, bias="bf16", act="silu", residual=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(25, 8300, 288), (45, 8300, 1056), (500, 1030, 96), (1100, 2300, 224)])
def test_more_than_a_round_of_small_tiles(fmt, dtype, M, N, K):
    run(M + K, M, N, K, fmt, dtype, bias="f32", act="relu", residual=True, drop=0.25)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(5, 50, 96), (200, 264, 256), (520, 640, 128)])
def test_epilogues(act, dtype, M, N, K):
    for i, (bias, drop, residual, keep_z) in enumerate([(None, 0.0, False, False), ("f32", 0.5, False, True),
                                                        ("bf16", 0.0, True, True), ("f32", 0.1, True, False)]):
        run(i, M, N, K, "mxfp8", dtype, bias, act, drop, residual, keep_z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(7, 61, 96), (40, 128, 64), (300, 333, 256)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 0), (8, 8), (5, 1)])
def test_strides_and_alignment(dtype, M, N, K, pad, shift):
    run(pad + shift, M, N, K, "mxfp4", dtype, "bf16", "silu", 0.25, True, True, pad, shift)
    run(pad + shift, M, N, K, "nvfp4", dtype, None, "none", 0.0, False, False, pad, shift, in_place=True)


@pytest.mark.parametrize("M,N", [(0, 5), (5, 0), (3, 40), (300, 264)])
def test_nothing_to_sum(M, N):
    W = mx.empty(mx.FORMATS["mxfp8"], N, 0, dev())
    x = torch.empty(M, 0, dtype=torch.bfloat16, device=dev())
    b = torch.arange(N, device=dev()).float()
    r, out = torch.ones(M, N, device=dev()), torch.full((M, N), 7.0, device=dev())
    mx.mx_linear(x, W, out, bias=b, act=mx.MX_ACT_RELU, residual=r)
    assert torch.equal(out, b.expand(M, N) + 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 300])
def test_extreme_weights(fmt, M):
    """Blocks of zeros at the smallest scale, one NaN scale, the largest codes."""
    g = np.random.default_rng(1)
    N, K = 40, 256
    codes, scales, ts = random_weights(g, fmt, N, K)
    codes[:8], scales[:8] = 0, 0
    codes[8] = {"mxfp4": 0x77, "nvfp4": 0x77, "mxfp8": 0x7E, "mxfp8_e5m2": 0x7B, "mxint8": 0x80}[fmt]
    scales[9, 1] = 0x7F if fmt == "nvfp4" else 255
    x, x64 = matrix(g.normal(size=(M, K)), "bf16")
    out = torch.empty(M, N, device=dev())
    mx.mx_linear(x, upload(fmt, codes, scales, ts), out)
    assert torch.isnan(out[:, 9]).all() and not torch.isnan(out[:, :9]).any() and not torch.isnan(out[:, 10:]).any()
    assert (out[:, :8] == 0).all()
    keep = [n for n in range(N) if n != 9]
    w = R.weights(fmt, codes, scales, 1.0 if ts is None else ts)[keep]
    _, (want, tol) = R.linear(x64, w, None, "none", None, None, "f32")
    check(out[:, keep], want, tol, fmt)


@pytest.mark.parametrize("fmt,lo,hi", [("mxfp4", 10, 239), ("mxfp8", 10, 239), ("mxfp8_e5m2", 10, 239),
                                       ("mxint8", 10, 254)])
def test_scale_codes_of_the_range(fmt, lo, hi):
    """One element of one column at each scale code, against a token of 1s."""
    v = {"mxfp4": (0x01, 0.5), "mxfp8": (0x09, 2.0 ** -6 * 1.125), "mxfp8_e5m2": (0x05, 2.0 ** -14 * 1.25),
         "mxint8": (0xC5, -59 / 64)}[fmt]
    n = hi - lo + 1
    codes = np.zeros((n, 16 if fmt == "mxfp4" else 32), np.uint8)
    codes[:, 3] = v[0]
    scales = np.arange(lo, hi + 1, dtype=np.uint8)[:, None]
    want = v[1] * 2.0 ** (np.arange(lo, hi + 1) - 127.0)
    for M in (1, 300):
        x = torch.ones(M, 32, dtype=torch.bfloat16, device=dev())
        out = torch.empty(M, n, device=dev())
        mx.mx_linear(x, upload(fmt, codes, scales, None), out)
        got = out.double().cpu().numpy()
        normal = np.abs(want) >= 2.0 ** -126
        assert (got[:, normal] == want[normal]).all()


def test_infinite_and_nan_tokens_stay_in_their_rows():
    g = np.random.default_rng(2)
    codes, scales, ts = random_weights(g, "mxfp8", 72, 160)
    for M in (5, 40, 300):
        x, _ = matrix(g.normal(size=(M, 160)), "bf16")
        clean = torch.empty(M, 72, device=dev())
        W = upload("mxfp8", codes, scales, ts)
        mx.mx_linear(x, W, clean)
        x[1, 159], x[3, 0] = float("nan"), float("inf")
        out = torch.empty(M, 72, device=dev())
        mx.mx_linear(x, W, out)
        assert torch.isnan(out[1]).all() and not torch.isfinite(out[3]).any()
        rest = [m for m in range(M) if m not in (1, 3)]
        assert torch.equal(out[rest], clean[rest])


def test_equal_calls_and_another_stream():
    x, W, b, r, out = run(5, 300, 264, 1056, "mxfp4", "f32", "f32", "gelu", 0.2, True)
    first = out.clone()
    side = torch.cuda.Stream()
    other = torch.empty_like(first)
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(bias=b, act=mx.MX_ACT_GELU, residual=r, drop=0.2, seed=2 ** 50 + 5, counter=2 ** 32 - 5)
    mx.mx_linear(x, W, other, stream=side, **kw)
    mx.mx_linear(x, W, out, **kw)
    torch.cuda.synchronize()
    assert torch.equal(first, out) and torch.equal(first, other)


def test_same_operands_as_the_quantizing_product():
    """z of quantized weights is mx_gemm_quantize_a's product where X is exact in
    8 bits: the same decoded operands."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-8, 9, (96, 256), generator=g, device=dev()).to(torch.bfloat16)
    x[:, ::32] = 8
    w = torch.randn(200, 256, generator=g, device=dev())
    W = mx.mx_quantize(w, mx.empty(mx.FORMATS["mxfp4"], 200, 256, dev()))
    a, b = torch.empty(96, 200, device=dev()), torch.empty(96, 200, device=dev())
    mx.mx_linear(x, W, a)
    mx.mx_gemm_quantize_a(x, mx.FORMATS["mxfp8"], W, b)
    torch.cuda.synchronize()
    scale = x.double().abs() @ w.double().abs().t() * 1.4
    assert ((a.double() - b.double()).abs() <= 2e-5 * scale).all()
