"""The combination of routed rows and its gradients against their 64-bit
definitions.  FP32 sums of k products: (k + 1) 2^-24 sum |w y|; the weights'
gradient: a lane adds 8 products for every 2048 columns, a tree of 10 levels
follows; outputs round once."""
import numpy as np
import pytest
import torch

from tests import moe_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def matrix(rows, cols, kind, fill=None, pad=0):
    unit = 16 // DT[kind].itemsize
    t = torch.full((rows, -(-cols // unit) * unit + pad), 7.0, dtype=DT[kind], device=dev())
    if fill is not None:
        t[:, :cols] = torch.from_numpy(fill.astype(np.float32)).to(dev())
    return t[:, :cols]


def host(t):
    return t.detach().cpu().double().numpy()


def slots(T, k, rows, seed, holes=0.2):
    g = np.random.default_rng([seed, T, k])
    s = g.permutation(rows)[: T * k].reshape(T, k) if rows >= T * k else g.integers(0, rows, (T, k))
    s = np.where(g.random((T, k)) < holes, -1, s)
    if T > 2:
        s[1] = -1                         # a token without a row
    return s, g


CASES = [(1, 8, 7168, 0), (1, 1, 1, 0), (5, 3, 8, 0), (33, 2, 65, 0), (40, 8, 519, 8), (70, 9, 1000, 0),
         (17, 20, 2056, 16), (129, 4, 512, 0), (6, 8, 4100, 0)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,cols,pad", CASES)
def test_forward(T, k, cols, pad, kind):
    s, g = slots(T, k, T * k + 3, 1)
    y = matrix(T * k + 3, cols, kind, g.standard_normal((T * k + 3, cols)), pad)
    unnamed = np.setdiff1d(np.arange(T * k + 3), s)
    y[torch.from_numpy(unnamed).to(dev())] = np.nan      # rows that no slot names are not read
    w = g.random((T, k)).astype(np.float32)
    w[s < 0] = np.nan                                    # nor are the weights of empty slots
    st, wt = torch.from_numpy(s.astype(np.int32)).to(dev()), torch.from_numpy(w).to(dev())
    for weights, okind, opad in ((wt, kind, pad), (None, "f32", 0), (wt, "bf16", 1)):
        out = matrix(T, cols, okind, pad=opad)
        mx.mx_combine(y, st, weights, out)
        torch.cuda.synchronize()
        want, mag = moe_ref.combine(host(y), s, np.ones((T, k)) if weights is None else w.astype(np.float64))
        tol = (k + 1) * U * mag + (2.0 ** -8 * np.abs(want) if okind == "bf16" else U * np.abs(want))
        assert np.all(np.abs(host(out) - want) <= tol)
        assert bool((out._base[:, cols:] == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,cols,pad", CASES)
def test_backward(T, k, cols, pad, kind):
    rows = T * k + 3
    s, g = slots(T, k, rows, 2)
    y = matrix(rows, cols, kind, g.standard_normal((rows, cols)), pad)
    do = matrix(T, cols, kind, g.standard_normal((T, cols)), pad)
    w = g.random((T, k)).astype(np.float32)
    w[s < 0] = np.nan
    st, wt = torch.from_numpy(s.astype(np.int32)).to(dev()), torch.from_numpy(w).to(dev())
    named = s >= 0
    t_of, j_of = np.nonzero(named)
    want_dw, mag = np.zeros((T, k)), np.zeros((T, k))
    yh, dh = host(y), host(do)
    want_dw[named] = (dh[t_of] * yh[s[named]]).sum(1)
    mag[named] = np.abs(dh[t_of] * yh[s[named]]).sum(1)
    for want_rows, want_weights, weights in ((True, True, wt), (True, False, wt), (False, True, wt),
                                             (True, True, None)):
        dy = matrix(rows, cols, kind, pad=pad) if want_rows else None
        dw = torch.full((T, k), 7.0, device=dev()) if want_weights else None
        mx.mx_combine_backward(do, y if want_weights else None, st, weights, dy, dw)
        torch.cuda.synchronize()
        if want_weights:
            n = 8 * -(-cols // 2048) + 12
            assert np.all(np.abs(host(dw) - want_dw) <= n * U * mag)
        if want_rows:
            want = np.full((rows, cols), 7.0)            # rows without a slot keep what they held
            ww = np.ones((T, k)) if weights is None else w.astype(np.float64)
            want[s[named]] = ww[named][:, None] * dh[t_of]
            tol = (2.0 ** -8 if kind == "bf16" else U) * np.abs(want)
            assert np.all(np.abs(host(dy) - want) <= tol)
            assert bool((dy._base[:, cols:] == 7.0).all())


def test_rows_past_the_matrix_add_nothing():
    y = matrix(4, 16, "f32", np.ones((4, 16)))
    s = torch.tensor([[0, 4], [1 << 30, 3]], dtype=torch.int32, device=dev())
    out, dw = matrix(2, 16, "f32"), torch.full((2, 2), 7.0, device=dev())
    mx.mx_combine(y, s, None, out)
    dy = matrix(4, 16, "f32")
    mx.mx_combine_backward(out, y, s, None, dy, dw)
    torch.cuda.synchronize()
    assert bool((out == 1).all())
    assert torch.equal(dw.cpu(), torch.tensor([[16.0, 0.0], [0.0, 16.0]]))
    assert bool((dy[1:3] == 7).all()) and bool((dy[0] == 1).all()) and bool((dy[3] == 1).all())


def test_gradients_against_differences():
    """f = <d_out, combine>: linear in Y and in w, so difference quotients are
    exact up to rounding (1e-16 / h in 64 bits); FP32 leaves 1e-5."""
    T, k, cols = 3, 2, 10
    s, g = slots(T, k, T * k, 3, holes=0.0)
    y, do, w = (g.standard_normal(n) for n in ((T * k, cols), (T, cols), (T, k)))
    yt, dot = matrix(T * k, cols, "f32", y), matrix(T, cols, "f32", do)
    wt = torch.from_numpy(w.astype(np.float32)).to(dev())
    st = torch.from_numpy(s.astype(np.int32)).to(dev())
    dy, dw = matrix(T * k, cols, "f32", np.zeros((T * k, cols))), torch.empty(T, k, device=dev())
    mx.mx_combine_backward(dot, yt, st, wt, dy, dw)
    torch.cuda.synchronize()
    f = lambda a, b: (moe_ref.combine(a, s, b)[0] * do).sum()
    h = 1e-3
    for i in np.ndindex(*y.shape):
        a, b = y.copy(), y.copy()
        a[i] += h
        b[i] -= h
        assert abs(float(dy[i]) - (f(a, w) - f(b, w)) / (2 * h)) <= 1e-5
    for i in np.ndindex(*w.shape):
        a, b = w.copy(), w.copy()
        a[i] += h
        b[i] -= h
        assert abs(float(dw[i]) - (f(y, a) - f(y, b)) / (2 * h)) <= 1e-5


def test_repeats_bit_for_bit_and_on_another_stream():
    T, k, cols = 300, 8, 1024
    s, g = slots(T, k, T * k, 4)
    y, do = matrix(T * k, cols, "bf16", g.standard_normal((T * k, cols))), matrix(T, cols, "bf16", g.standard_normal((T, cols)))
    st, wt = torch.from_numpy(s.astype(np.int32)).to(dev()), torch.from_numpy(g.random((T, k)).astype(np.float32)).to(dev())
    stream = torch.cuda.Stream()
    got = []
    for i in range(4):
        out, dw = matrix(T, cols, "bf16"), torch.empty(T, k, device=dev())
        stream.wait_stream(torch.cuda.current_stream())
        use = stream if i % 2 else None
        mx.mx_combine(y, st, wt, out, stream=use)
        mx.mx_combine_backward(do, y, st, wt, None, dw, stream=use)
        torch.cuda.synchronize()
        got.append((out, dw))
    for out, dw in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(dw, got[0][1])
