"""The router against its 64-bit definition: choices, order and counts exactly,
weights, sums, loss and gradients within bounds.

Bounds (u = 2^-24): exp2 of a rounded product has relative error at most
4 u (1 + |x - max|) + 2^-22 (the instruction is good to one unit), quotients
and the sum over E experts add a few u more, so p is within
E_P = u (16 + 4 span + E / 8) with span the largest max - x in play (a lane
adds E / 16 terms or fewer, then a tree).  Sums over tokens run in chains of at
most per / 8 + 8 + 256 terms."""
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


def scores(T, E, kind, seed, std=1.5, pad=0):
    g = np.random.default_rng([seed, T, E])
    x = (g.standard_normal((T, E)) * std + 0.5 * g.standard_normal(E)).astype(np.float32)
    t = torch.zeros(T, E + pad, dtype=DT[kind], device=dev())
    t[:, :E] = torch.from_numpy(x).to(dev())
    return t[:, :E]


def host(t):
    return t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def forward(x, topk, mask=None, normalize=False):
    r = mx.routing(x.shape[0], x.shape[1], topk, device=dev())
    for n in ("experts", "weights", "slot_row", "row_index", "group_offsets", "counts", "valid", "prob_sum", "loss"):
        getattr(r, n).fill_(77)
    r.workspace.fill_(0xA5)
    m = None if mask is None else torch.from_numpy(mask.astype(np.uint8)).to(dev())
    mx.mx_route(x, r, token_mask=m, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    torch.cuda.synchronize()
    return r, m


def check_forward(x, topk, mask=None, normalize=False):
    r, m = forward(x, topk, mask, normalize)
    T, E = x.shape
    want = moe_ref.route(host(x), topk, mask, normalize)
    for n in ("experts", "slot_row", "row_index", "group_offsets", "counts"):
        assert np.array_equal(host(getattr(r, n)), want[n]), n
    assert int(r.valid) == want["valid"]
    live = host(x) if mask is None else host(x)[mask != 0]
    f = np.isfinite(live)
    span = float(np.ptp(live[f])) if f.any() else 0.0
    ep = U * (16 + 4 * span + E / 8)
    assert np.all(np.abs(host(r.weights) - want["weights"]) <= 2 * ep * want["weights"] + 1e-37)
    chain = U * (T / 8 + 8 + 256)
    assert np.all(np.abs(host(r.prob_sum) - want["prob_sum"]) <= (ep + chain) * want["prob_sum"] + 1e-37)
    assert abs(float(r.loss) - want["loss"]) <= (ep + chain + U * (E + 16)) * want["loss"]
    return r, m, want, ep


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,topk", [
    (1, 1, 1), (1, 32, 8), (3, 2, 2), (5, 16, 1), (17, 17, 3), (63, 33, 4), (64, 64, 8), (65, 60, 6), (130, 100, 8),
    (200, 128, 7), (77, 129, 16), (300, 256, 8), (70, 257, 5), (129, 511, 8), (66, 512, 10), (65, 1000, 16),
    (90, 1024, 2)])
def test_forward(T, E, topk, kind):
    for normalize in (False, True):
        check_forward(scores(T, E, kind, 1), topk, normalize=normalize)


@pytest.mark.parametrize("T,E,topk", [(4097, 32, 8), (16448, 8, 2), (20000, 40, 6)])
def test_many_tokens(T, E, topk):
    """More than one block of tokens, and (past 16384) more than 64 tokens a block."""
    mask = np.random.default_rng(2).random(T) > 0.2
    check_forward(scores(T, E, "bf16", 3), topk, mask=mask.astype(np.uint8), normalize=True)


@pytest.mark.parametrize("E", [5, 24, 256, 300])
def test_masks_and_unchoosable_experts(E):
    T, topk = 150, 4
    g = np.random.default_rng(E)
    x = scores(T, E, "f32", 4)
    x[torch.from_numpy(g.random((T, E)) < 0.5).to(dev())] = -np.inf
    x[3] = -np.inf                       # a token without any expert
    x[4] = -np.inf
    x[4, E - 1] = -3.0e38                # one expert, at the type's low end
    x[5] = torch.finfo(torch.float32).min  # all equal, all at the lowest finite value
    mask = (g.random(T) > 0.3).astype(np.uint8)
    mask[3:6] = 1
    mask[10:12] = 0
    x[10], x[11] = np.nan, np.inf        # padding is not looked at
    check_forward(x, topk, mask)
    check_forward(x, topk, mask, normalize=True)
    check_forward(x, topk, np.zeros(T, np.uint8))  # nothing but padding


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ties_go_to_the_lower_index(kind):
    for E in (7, 32, 200, 700):
        x = scores(90, E, kind, 5)
        x[:, :] = (x * 1.5).round()      # few distinct values
        x[7] = 0.0
        check_forward(x, min(E, 8))


def test_nan_and_infinity_in_a_row():
    T, E, topk = 70, 40, 5
    x = scores(T, E, "f32", 6)
    x[2, 7], x[9, 0], x[11] = np.nan, np.inf, np.nan
    r, _ = forward(x, topk)
    want = moe_ref.route(host(x), topk)
    for n in ("experts", "slot_row", "row_index", "group_offsets", "counts"):
        assert np.array_equal(host(getattr(r, n)), want[n]), n
    w = host(r.weights)
    assert np.isnan(w[2]).all() and np.isnan(w[9]).all() and (w[11] == 0).all()
    assert np.isfinite(np.delete(w, [2, 9, 11], 0)).all()
    assert np.isnan(host(r.prob_sum)).any() and np.isnan(float(r.loss))
    r, _ = forward(x, topk, normalize=True)
    assert np.isnan(host(r.weights)[2]).all() and np.isnan(host(r.weights)[9]).all()


def test_row_pitch_and_alignment():
    for kind in DT:
        for pad in (1, 3, 8):
            check_forward(scores(80, 60, kind, 7, pad=pad), 6)
    base = scores(80, 61, "f32", 8)
    check_forward(base[:, 1:], 6)        # rows start at any element


def test_no_tokens():
    r, _ = forward(torch.empty(0, 12, device=dev()), 3)
    assert not host(r.group_offsets).any() and not host(r.counts).any() and not host(r.prob_sum).any()
    assert int(r.valid) == 0 and float(r.loss) == 0.0


def backward(x, r, m, dw, dl, normalize, pad=0):
    T, E = x.shape
    full = torch.full((T, E + pad), 7.0, dtype=x.dtype, device=dev())
    mx.mx_route_backward(x, r, dw, dl, full[:, :E], token_mask=m, flags=mx.MX_ROUTE_NORMALIZE if normalize else 0)
    torch.cuda.synchronize()
    assert bool((full[:, E:] == 7.0).all())
    return full[:, :E]


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,topk,pad", [(1, 32, 8, 0), (7, 1, 1, 0), (65, 33, 4, 1), (130, 128, 16, 0),
                                          (99, 256, 8, 8), (40, 500, 6, 0), (33, 1024, 3, 0)])
def test_backward(T, E, topk, pad, kind, normalize):
    g = np.random.default_rng(T)
    x = scores(T, E, kind, 9)
    if E > topk + 2:
        x[0, 2] = -np.inf
    mask = (g.random(T) > 0.2).astype(np.uint8)
    mask[0] = 1
    r, m, want, ep = check_forward(x, topk, mask, normalize)
    dw = torch.from_numpy(g.standard_normal((T, topk)).astype(np.float32)).to(dev())
    dl = torch.tensor([0.7], device=dev())
    for a, b in ((dw, dl), (dw, None), (None, dl)):
        got = host(backward(x, r, m, a, b, normalize, pad))
        d, size = moe_ref.route_backward(want["p"], want["experts"], want["counts"], want["valid"],
                                         np.zeros((T, topk)) if a is None else host(a),
                                         0.0 if b is None else float(b), normalize)
        tol = (4 * ep + 32 * U) * size + 1e-37
        if kind == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(d) + 1e-38
        assert np.all(np.abs(got - d) <= tol)
        assert not got[mask == 0].any()


@pytest.mark.parametrize("normalize", [False, True])
def test_backward_against_differences(normalize):
    """Difference quotients of the 64-bit objective: relative truncation error
    h^2 / 6 times third derivatives of order 1, rounding 1e-16 / h: with
    h = 1e-4, 1e-7 of the gradient's scale covers both and FP32's 1e-6."""
    T, E, topk = 9, 12, 3
    x = scores(T, E, "f32", 10)
    g = np.random.default_rng(1)
    dw, dl = g.standard_normal((T, topk)), 0.9
    r, m, want, _ = check_forward(x, topk, normalize=normalize)
    dw32 = torch.from_numpy(dw.astype(np.float32)).to(dev())
    got = host(backward(x, r, m, dw32, torch.tensor([dl], device=dev()), normalize))
    f = lambda y: moe_ref.route_objective(y, want["experts"], want["counts"], T, host(dw32), float(np.float32(dl)),
                                          normalize)
    x64, h = host(x), 1e-4
    for t in range(T):
        for e in range(E):
            a, b = x64.copy(), x64.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs(got[t, e] - (f(a) - f(b)) / (2 * h)) <= 5e-6


def test_global_counts_scale_the_loss_gradient():
    """counts and valid summed over two devices: the gradient of the common loss."""
    T, E, topk = 40, 16, 2
    xa, xb = scores(T, E, "f32", 11), scores(T, E, "f32", 12)
    both = moe_ref.route(np.concatenate([host(xa), host(xb)]), topk)
    r, m, want, ep = check_forward(xa, topk)
    r.counts.copy_(torch.from_numpy(both["counts"]))
    r.valid.fill_(2 * T)
    got = host(backward(xa, r, m, None, torch.tensor([1.0], device=dev()), False))
    d, size = moe_ref.route_backward(want["p"], want["experts"], both["counts"], 2 * T, np.zeros((T, topk)), 1.0,
                                     False)
    assert np.all(np.abs(got - d) <= (4 * ep + 32 * U) * size)


def test_repeats_bit_for_bit_and_on_another_stream():
    x = scores(3000, 64, "f32", 13)
    r0, _ = forward(x, 6)
    keep = {n: getattr(r0, n).clone() for n in ("experts", "weights", "slot_row", "row_index", "prob_sum", "loss")}
    s = torch.cuda.Stream()
    for _ in range(5):
        r = mx.routing(3000, 64, 6, device=dev())
        s.wait_stream(torch.cuda.current_stream())
        mx.mx_route(x, r, stream=s)
        s.synchronize()
        for n, v in keep.items():
            assert torch.equal(getattr(r, n), v), n
