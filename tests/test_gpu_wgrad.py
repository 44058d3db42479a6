"""The grouped weight gradient from an 8-bit checkpoint against the 64-bit
product of the decoded values.  Products of BF16 values are exact in FP32, so
the error is that of FP32 sums of n terms, at most n 2^-24 sum |a b| in any
order (the instruction's own adds included: 2^-23 per term is allowed), plus
half a unit of the output's type."""
import numpy as np
import pytest
import torch

from tests import moe_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(rows, groups, N, K, fmt, seed, gather=False, empty=()):
    g = np.random.default_rng([seed, rows, groups, N, K])
    share = g.random(groups) + 0.05
    share[list(empty)] = 0
    cuts = np.round(np.cumsum(share) / share.sum() * rows).astype(np.int64)
    offsets = np.concatenate([[0], cuts])
    x_rows = max(rows // 3, 1) if gather else rows
    x = torch.from_numpy(g.standard_normal((x_rows, K)).astype(np.float32)).to(dev())
    x[:, : K // 8] *= 20
    X = mx.empty(mx.FORMATS[fmt], x_rows, K, dev())
    if x_rows:
        mx.mx_quantize(x, X)
    pitch = (N + 7) // 8 * 8 + (8 if seed % 2 else 0)
    dy = torch.full((rows, pitch), np.nan, dtype=torch.bfloat16, device=dev())[:, :N]
    dy.copy_(torch.from_numpy(g.standard_normal((rows, N)).astype(np.float32)))
    index = torch.from_numpy(g.integers(0, x_rows, rows).astype(np.int32)).to(dev()) if gather else None
    return dy, X, index, torch.from_numpy(offsets).to(dev())


def decoded(X):
    out = torch.empty(X.rows, X.cols, device=dev())
    if X.rows:
        mx.mx_dequantize(X, out)
    return out.cpu().double().numpy()


def check(dy, X, index, offsets, kind, pad=0, accumulate=False, groups=None):
    groups = groups or offsets.numel() - 1
    N, K = dy.shape[1], X.cols
    full = torch.full((groups * N, K + pad), 3.0, dtype=DT[kind], device=dev())
    dw = full[:, :K]
    mx.mx_wgrad_grouped(dy, X, index, groups, offsets, dw, flags=mx.MX_WGRAD_ACCUMULATE if accumulate else 0)
    torch.cuda.synchronize()
    off = [0, dy.shape[0]] if offsets is None else offsets.tolist()
    want, mag, n = moe_ref.wgrad(dy.cpu().double().numpy(), decoded(X), off,
                                 None if index is None else index.cpu().numpy())
    tol = (n.repeat(N)[:, None] + 2) * 2.0 ** -23 * mag
    if accumulate:
        want = want + 3.0
        tol = tol + 2.0 ** -23 * np.abs(want)
    if kind == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want)
    got = dw.cpu().double().numpy()
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))
    assert bool((full[:, K:] == 3.0).all())


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp8_e5m2", "mxint8"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,N,K", [(1, 1, 8, 32), (31, 3, 1, 32), (100, 5, 129, 160), (257, 2, 136, 288),
                                             (64, 70, 33, 64), (1000, 4, 264, 544)])
def test_small(rows, groups, N, K, kind, fmt):
    for gather in (False, True):
        check(*case(rows, groups, N, K, fmt, rows + gather, gather), kind)


@pytest.mark.parametrize("rows,groups,N,K", [(2000, 3, 512, 1024), (1500, 2, 1032, 800), (4100, 1, 300, 2048)])
def test_larger_tiles(rows, groups, N, K):
    for fmt in ("mxfp8", "mxint8"):
        check(*case(rows, groups, N, K, fmt, 1, True), "f32")
        check(*case(rows, groups, N, K, fmt, 2), "bf16")


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp8_e5m2", "mxint8"])
@pytest.mark.parametrize("rows,groups,N,K", [(5000, 64, 264, 512), (3000, 140, 256, 288), (9000, 70, 392, 512)])
def test_many_tiles(rows, groups, N, K, fmt):
    """Enough tiles of 256 x 256 for the larger ones, one or several a workgroup;
    groups of no, a few and many steps of rows, tiles that lie partly outside."""
    for gather in (False, True):
        args = case(rows, groups, N, K, fmt, 11 + gather, gather, empty=(0, 5, groups - 1))
        check(*args, "bf16" if gather else "f32")
        check(*args, "f32" if gather else "bf16", pad=5, accumulate=True)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("rows,groups,N,K,empty", [(8192, 1, 64, 128, ()), (5000, 3, 129, 160, (1,)),
                                                   (6000, 7, 40, 288, (0, 2, 6)), (20000, 70, 16, 96, (0, 64, 69)),
                                                   (150000, 70, 16, 96, (0, 64, 69)),
                                                   (3001, 2, 264, 512, ()), (9000, 5, 1, 64, (4,))])
def test_few_tiles_and_many_rows(rows, groups, N, K, empty, fmt):
    """The rows of a group are summed in parts: groups of one part, of many, of
    none."""
    assert (rows, groups) == (20000, 70) or mx.mx_wgrad_workspace_bytes(rows, N, K, groups) > 0
    for gather in (False, True):
        args = case(rows, groups, N, K, fmt, 21 + gather, gather, empty=empty)
        check(*args, "bf16" if gather else "f32")
        check(*args, "f32" if gather else "bf16", pad=5, accumulate=True)


@pytest.mark.parametrize("rows,groups,N,K,fmt", [(32768, 1, 2048, 2048, "mxfp8"), (32768, 4, 1024, 1056, "mxint8"),
                                                 (20000, 3, 1032, 1024, "mxfp8_e5m2")])
def test_parts_of_large_tiles(rows, groups, N, K, fmt):
    """Parts where the larger tiles are chosen (the reference on the GPU)."""
    assert mx.mx_wgrad_workspace_bytes(rows, N, K, groups) > 0
    g = torch.Generator(device="cuda").manual_seed(rows + groups)
    X = mx.empty(mx.FORMATS[fmt], rows, K, dev())
    mx.mx_quantize(torch.randn(rows, K, generator=g, device=dev()), X)
    x = torch.empty(rows, K, device=dev())
    mx.mx_dequantize(X, x)
    dy = torch.randn(rows, N, generator=g, device=dev()).to(torch.bfloat16)
    cuts = [0] + sorted(torch.randint(0, rows, (groups - 1,), generator=g, device=dev()).tolist()) + [rows]
    off = None if groups == 1 else torch.tensor(cuts, dtype=torch.int64, device=dev())
    index = torch.randperm(rows, generator=g, device=dev()).int()
    for idx in (None, index):
        dw = torch.empty(groups * N, K, device=dev())
        mx.mx_wgrad_grouped(dy, X, idx, groups, off, dw)
        src = x if idx is None else x[idx.long()]
        for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
            d, v = dy[a:b].double().t().contiguous(), src[a:b].double()
            tol = (b - a + 2) * 2.0 ** -23 * (d.abs() @ v.abs())
            assert ((dw[e * N:(e + 1) * N].double() - d @ v).abs() <= tol).all(), e


def test_parts_with_offsets_that_break_their_contract_and_repeats():
    dy, X, _, _ = case(6000, 4, 64, 128, "mxfp8", 23)
    for off in ([-5, 4000, 3000, 9000, 6000], [5000, 6000, 2000, 2000, 1 << 40], [-1, -1, -1, -1, -1],
                [6000, 0, 6000, 0, 6000], [0, 6000, 0, 6000, 0]):
        at = torch.tensor(off, dtype=torch.int64, device=dev())
        outs = []
        ws = torch.full((mx.mx_wgrad_workspace_bytes(6000, 64, 128, 4),), 0xFF, dtype=torch.uint8, device=dev())
        for w in (ws, None, ws):
            dw = torch.full((4 * 64, 128), 3.0, device=dev())
            mx.mx_wgrad_grouped(dy, X, None, 4, at, dw, workspace=w)
            torch.cuda.synchronize()
            outs.append(dw)
        assert all(torch.equal(o, outs[0]) for o in outs)
        a, x = dy.cpu().double().numpy(), decoded(X)
        for e in range(4):
            lo = min(max(off[e], 0), 6000)
            hi = min(max(off[e + 1], lo), 6000)
            assert np.allclose(outs[0][64 * e : 64 * e + 64].cpu().numpy(), a[lo:hi].T @ x[lo:hi], rtol=1e-4, atol=2e-2)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("rows,groups,N,K", [(9000, 20, 1032, 1024), (6000, 33, 776, 1056), (3000, 36, 640, 576),
                                             (4000, 45, 33, 2112)])
def test_tiles_of_a_workgroup_at_other_columns(rows, groups, N, K, fmt):
    """Several tiles a workgroup, each at other columns than the one before."""
    for gather in (False, True):
        check(*case(rows, groups, N, K, fmt, 31 + gather, gather, empty=(3, groups - 2)), "bf16" if gather else "f32")


def test_many_tiles_nan_scale_row_index_and_repeats():
    dy, X, index, off = case(4000, 64, 264, 512, "mxfp8", 13, True)
    lo, hi = int(off[9]), int(off[10])
    assert hi > lo
    X.scales[int(index[lo]), 2] = 0xFF
    index[lo + 1 :][index[lo + 1 :] == index[lo]] = (int(index[lo]) + 1) % X.rows
    index[:lo][index[:lo] == index[lo]] = (int(index[lo]) + 1) % X.rows
    outs = []
    for _ in range(3):
        dw = torch.empty(64 * 264, 512, device=dev())
        mx.mx_wgrad_grouped(dy, X, index, 64, off, dw)
        torch.cuda.synchronize()
        outs.append(dw)
    bad = torch.isnan(outs[0]).cpu().numpy()
    want = np.zeros_like(bad)
    want[9 * 264 : 10 * 264, 64:96] = True
    assert np.array_equal(bad, want)
    assert all(torch.equal(o.nan_to_num(7.0), outs[0].nan_to_num(7.0)) for o in outs)


def test_groups_without_rows_and_accumulation():
    for kind in DT:
        for gather in (False, True):
            args = case(300, 7, 72, 96, "mxfp8", 4, gather, empty=(0, 3, 6))
            check(*args, kind)
            check(*args, kind, pad=5, accumulate=True)


def test_one_group_without_offsets_and_no_rows():
    dy, X, index, _ = case(150, 1, 40, 64, "mxint8", 5)
    check(dy, X, index, None, "f32", groups=1)
    dy, X, index, off = case(0, 3, 40, 64, "mxfp8", 6)
    check(dy, X, index, off, "f32")


def test_offsets_that_break_their_contract_stay_in_bounds():
    dy, X, _, _ = case(64, 3, 32, 64, "mxfp8", 7)
    off = torch.tensor([-5, 40, 20, 900], dtype=torch.int64, device=dev())
    dw = torch.empty(96, 64, device=dev())
    mx.mx_wgrad_grouped(dy, X, None, 3, off, dw)
    torch.cuda.synchronize()
    a, x = dy.cpu().double().numpy(), decoded(X)
    want = np.concatenate([a[:40].T @ x[:40], np.zeros((32, 64)), a[20:].T @ x[20:]])
    assert np.allclose(dw.cpu().numpy(), want, rtol=1e-4, atol=1e-3)


def test_row_index_is_clamped():
    dy, X, index, off = case(50, 2, 32, 64, "mxfp8", 8, True)
    bad = index.clone()
    bad[3], bad[7] = -9, 1 << 30
    fixed = bad.clamp(0, X.rows - 1)
    out = [torch.empty(64, 64, device=dev()) for _ in range(2)]
    mx.mx_wgrad_grouped(dy, X, bad, 2, off, out[0])
    mx.mx_wgrad_grouped(dy, X, fixed, 2, off, out[1])
    torch.cuda.synchronize()
    assert torch.equal(*out)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp8_e5m2", "mxint8"])
def test_nan_scale_reaches_its_columns_of_its_group_only(fmt):
    dy, X, _, off = case(90, 3, 40, 128, fmt, 9)
    lo, hi = int(off[1]), int(off[2])
    assert hi > lo
    X.scales[lo, 2] = 0xFF
    dw = torch.empty(120, 128, device=dev())
    mx.mx_wgrad_grouped(dy, X, None, 3, off, dw)
    torch.cuda.synchronize()
    bad = torch.isnan(dw).cpu().numpy()
    want = np.zeros_like(bad)
    want[40:80, 64:96] = True
    assert np.array_equal(bad, want)


def test_extreme_scales():
    """Codes whose values BF16 holds only rounded (E4M3 below scale code 3) or
    at the top of its range."""
    rows, N, K = 16, 16, 32
    for fmt, codes in (("mxfp8", (0, 1, 3, 240)), ("mxint8", (10, 200, 240))):
        for sc in codes:
            X = mx.empty(mx.FORMATS[fmt], rows, K, dev())
            X.codes.copy_(torch.arange(rows * K, dtype=torch.int32).view(rows, K) % 120)
            X.scales.fill_(sc)
            dy = torch.ones(rows, N, dtype=torch.bfloat16, device=dev())
            dw = torch.empty(N, K, device=dev())
            mx.mx_wgrad_grouped(dy, X, None, 1, None, dw)
            torch.cuda.synchronize()
            want = decoded(X).sum(0)[None].repeat(N, 0)
            assert np.all(np.abs(dw.cpu().double().numpy() - want) <= 2.0 ** -19 * np.abs(want) + rows * 2.0 ** -133)


def test_gradient_against_differences():
    """f(W) = sum over the rows r of group e of <dY[r], W_e X[src(r)]> is linear
    in W, so its difference quotients in 64 bits are exact but for 2^-52 |f| /
    step, far below the bound of the kernel's sums."""
    dy, X, index, off = case(90, 3, 16, 64, "mxfp8", 14, True)
    dw = torch.empty(48, 64, device=dev())
    mx.mx_wgrad_grouped(dy, X, index, 3, off, dw)
    torch.cuda.synchronize()
    a, x, o = dy.cpu().double().numpy(), decoded(X)[index.cpu().numpy()], off.tolist()
    g = np.random.default_rng(1)
    W = g.standard_normal((3, 16, 64))

    def f(W):
        return sum(float(np.sum(a[o[e]:o[e + 1]] * (x[o[e]:o[e + 1]] @ W[e].T))) for e in range(3))

    for _ in range(20):
        e, n, k = g.integers(3), g.integers(16), g.integers(64)
        D = np.zeros_like(W)
        D[e, n, k] = 0.5
        mag = float(np.sum(np.abs(a[o[e]:o[e + 1], n] * x[o[e]:o[e + 1], k])))
        assert abs(float(dw[e * 16 + n, k]) - (f(W + D) - f(W - D))) <= 92 * 2.0 ** -23 * mag + 1e-9


def test_repeats_bit_for_bit_and_on_another_stream():
    dy, X, index, off = case(3000, 5, 264, 544, "mxfp8", 10, True)
    first = torch.empty(5 * 264, 544, device=dev())
    mx.mx_wgrad_grouped(dy, X, index, 5, off, first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(4):
        again = torch.empty_like(first)
        s.wait_stream(torch.cuda.current_stream())
        mx.mx_wgrad_grouped(dy, X, index, 5, off, again, stream=s)
        s.synchronize()
        assert torch.equal(again, first)
