"""mx_logprob and mx_logprob_backward against their formulas in 64 bits: sizes,
alignments, ties, entries and rows without probability, padding, in place."""
import numpy as np
import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev
    from tests.test_gpu_linear import matrix

INF, NAN = float("inf"), float("nan")


def same(got, want, tol, what):
    got = got.double().cpu().numpy()
    both = np.isnan(got) & np.isnan(want) | (got == want)
    with np.errstate(invalid="ignore"):
        bad = ~(both | (np.abs(got - want) <= tol))
    assert not bad.any(), (what, int(bad.sum()), [(tuple(i), got[tuple(i)], want[tuple(i)], tol[tuple(i)])
                                                  for i in np.argwhere(bad)[:4]])


def run(values, target, topk, scale=1.0, dtype="bf16", pad=0, shift=0, grads=True):
    T, V = values.shape
    x, x64 = matrix(values, dtype, pad, shift)
    to = lambda a: torch.from_numpy(np.asarray(a)).to(dev())
    at = None if target is None else to(np.asarray(target, np.int64))
    s = mx.logprobs(T, V, topk, dev())
    for t in (s.logp, s.entropy, s.row_max, s.log_sum, s.top_logp):
        t.fill_(77)
    s.top_id.fill_(77)
    mx.mx_logprob(x, at, s, scale)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want, tol = R.logprob(x64, target, scale, topk)
    for n in ("logp", "entropy", "row_max", "log_sum"):
        if n == "logp" and target is None:
            assert (s.logp == 77).all()
            continue
        if n in ("row_max", "log_sum"):
            ok = ~np.isnan(want[n])  # (of such rows the results are NaN, what is saved is not specified)
            same(getattr(s, n)[to(ok)], want[n][ok], tol[n][ok], n)
        else:
            same(getattr(s, n), want[n], tol[n], n)
    assert np.array_equal(s.top_id.cpu().numpy(), want["top_id"])
    same(s.top_logp, want["top_logp"], tol["top_logp"], "top_logp")
    if not grads:
        return s, x
    g = np.random.default_rng(T)
    dl, dh = (g.normal(size=T).astype(np.float32) for _ in range(2))
    dx = matrix(np.zeros((T, V)), dtype, pad, shift)[0]
    for a, b in ((dl, dh), (dl, None), (None, dh)):
        with np.errstate(invalid="ignore"):
            w, t = R.logprob_backward(x64, target, scale, a, b, tol, dtype)
        opt = lambda v: None if v is None else to(v)
        mx.mx_logprob_backward(x, at, s, opt(a), opt(b), dx, scale)
        same(dx, w, t, "d_logits")
        if pad:
            assert (dx.as_strided((T, pad), (V + pad, 1), shift + V) == 99).all()
    # an output of another alignment, and in place
    other = matrix(np.zeros((T, V)), dtype, pad + 1, shift + 1)[0]
    mx.mx_logprob_backward(x, at, s, opt(None), to(dh), other, scale)
    assert torch.equal(other.nan_to_num(7), dx.nan_to_num(7))
    mx.mx_logprob_backward(x, at, s, opt(None), to(dh), x, scale)
    assert torch.equal(x.nan_to_num(7), dx.nan_to_num(7))
    return s, x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,topk", [(1, 1, 1), (2, 2, 2), (3, 7, 5), (5, 8, 0), (4, 63, 20), (7, 64, 32), (3, 511, 1),
                                      (2, 513, 20), (6, 4097, 8), (3, 8191, 32), (2, 50257, 20), (1, 70001, 0),
                                      (1, 65536, 32), (5, 100003, 20), (100, 70000, 0), (64, 100000, 1), (140, 66000, 5)])
def test_sizes(dtype, T, V, topk):
    g = np.random.default_rng(T * V)
    run(g.normal(size=(T, V)) * 3, g.integers(0, V, T), topk, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (5, 3), (8, 8), (7, 7)])
def test_strides_and_alignment(dtype, pad, shift):
    g = np.random.default_rng(pad)
    run(g.normal(size=(9, 1000)) * 2, g.integers(0, 1000, 9), 6, 0.7, dtype, pad, shift)


@pytest.mark.parametrize("tokens", [64, 700, 3000])
def test_many_rows(tokens):
    g = np.random.default_rng(tokens)
    target = g.integers(-1, 300, tokens)
    run(g.normal(size=(tokens, 300)) * 4, target, 3, 1.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (5, 3)])
def test_rows_in_parts(dtype, pad, shift):
    """Few long rows: alternatives spread over the parts, all in one, parts without
    an entry, rows without any, padding."""
    V = 120001
    g = np.random.default_rng(shift)
    x = g.normal(size=(9, V)) * 2
    x[1, 40000:40040] = np.linspace(30, 40, 40)
    x[2, :70000] = -INF
    x[3] = -INF
    x[4] = -INF
    x[4, [5, 50000, V - 1]] = [1.0, 1.0, 2.0]
    x[5] = 0.25
    x[6, ::9000] = 20.0
    x[7, 80000] = NAN
    target = [0, 40039, V - 1, 3, 50000, 7, 9000, 1, -1]
    run(x, target, 32, 1.0, dtype, pad, shift)
    run(x, None, 4, 0.5, dtype, pad, shift)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two values", "zeros of both signs", "steps"])
@pytest.mark.parametrize("V", [2500, 20000, 110000])
def test_ties_and_orders(dtype, order, V):
    v = {"rising": np.linspace(-5, 5, V), "falling": np.linspace(5, -5, V), "equal": np.full(V, 1.5),
         "two values": np.where(np.arange(V) % 777 == 5, 2.0, 1.0),
         "zeros of both signs": np.where(np.arange(V) % 2 == 0, -0.0, 0.0), "steps": np.arange(V) // 640 % 5 * 1.0}[order]
    for topk in (1, 20, 32):
        run(np.stack([v, v[::-1].copy()]), [3, V - 1], topk, dtype=dtype, grads=topk == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 5000])
def test_entries_and_rows_without_probability(dtype, V):
    g = np.random.default_rng(V)
    x = g.normal(size=(12, V)) * 2
    x[1, g.random(V) < 0.9] = -INF
    x[2] = -INF                       # nothing left
    x[3] = -INF
    x[3, V - 2] = 4.0                 # one left
    x[4] = -3.3e38                    # the type's lowest values, alone
    x[5, ::2] = -3.3e38               # and as a mask
    x[6, 7] = NAN
    x[7, 9] = INF
    x[8] = 60000.0                    # large scores
    x[8, 3] = 60512.0
    x[9] *= 50                        # all but one vanish
    x[10] = -INF
    x[10, [3, 30]] = [-7.0, -7.0]
    x[11] = 0.0
    target = [0, 2, 1, V - 2, 5, 1, 3, 9, 3, int(np.argmax(x[9])), 30, V]
    for scale in (1.0, 3.0):
        run(x, target, 20, scale, dtype)
    run(x, None, 5, 1.0, dtype)


def test_sure_tokens():
    """log p close to 0 keeps an error near that of FP32 numbers around 1."""
    x = np.zeros((4, 1000))
    x[:, 5] = [10, 14, 17, 40]
    run(x, [5, 5, 5, 5], 2, 1.0, "f32")
    run(x, [5, 5, 0, 1], 2, 2.0, "f32")


def test_equal_calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(300, 9001, generator=g, device=dev()) * 3).to(torch.bfloat16)
    t = torch.randint(0, 9001, (300,), generator=g, device=dev())
    a, b = mx.logprobs(300, 9001, 20, dev()), mx.logprobs(300, 9001, 20, dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mx.mx_logprob(x, t, a)
    mx.mx_logprob(x, t, b, stream=side)
    torch.cuda.synchronize()
    for n in ("logp", "entropy", "row_max", "log_sum", "top_id", "top_logp"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_row_past_32_bit_offsets():
    T, V = 5, 1 << 29
    x = torch.zeros(T, V, dtype=torch.bfloat16, device=dev())
    x[:, 3] = 30.0
    x[4, V - 1] = 31.0
    t = torch.tensor([3, 3, 3, -5, V - 1], device=dev())
    s = mx.mx_logprob(x, t, mx.logprobs(T, V, 2, dev()))
    ls = np.log1p((V - 1) * np.exp(-30.0))
    # the lane that holds the 1 loses its other terms, 2^19 e^-30 or twice that; 10 joins of lanes and waves round
    np.testing.assert_allclose(s.logp[:3].cpu().numpy(), -ls, rtol=0, atol=2 ** 21 * np.exp(-30) + 12 * R.U)
    assert s.top_id.tolist() == [[3, 0], [3, 0], [3, 0], [-1, -1], [V - 1, 3]]
    d = mx.mx_logprob_backward(x, t, s, torch.ones(T, device=dev()), None, x)
    assert (d[3, ::65536] == 0).all() and float(d[4, V - 1]) > 0 > float(d[4, 3])
