"""Slots that name one row: the sum takes it as often as it is named, and the
gradient of the weights has its product with each token.  (The gradient of the
rows wants distinct rows, and distinct rows are what a routing gives.)  Bounds
as for distinct rows: (k + 1) 2^-24 sum |w y| for sums of k products, and
a chain and a tree of 8 ceil(cols / 2048) + 12 adds for the weights' gradient."""
import numpy as np
import pytest
import torch

from tests import moe_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import microscaling_precision_gemm_amd as mx
    from tests.gpu_util import dev

U = 2.0 ** -24


@pytest.mark.parametrize("T,k,cols,rows", [(1, 8, 64, 1), (9, 3, 520, 4), (700, 8, 1024, 50)])
def test_repeated_rows(T, k, cols, rows):
    g = np.random.default_rng(T)
    s, w = g.integers(-1, rows, (T, k)), g.random((T, k)).astype(np.float32)
    s[0] = 0  # one token, one row, in all of its slots
    y, do = (torch.from_numpy(g.standard_normal(n).astype(np.float32)).to(dev()) for n in ((rows, cols), (T, cols)))
    st, wt = torch.from_numpy(s.astype(np.int32)).to(dev()), torch.from_numpy(w).to(dev())
    out, dw = torch.empty(T, cols, device=dev()), torch.empty(T, k, device=dev())
    mx.mx_combine(y, st, wt, out)
    mx.mx_combine_backward(do, y, st, wt, None, dw)
    torch.cuda.synchronize()
    yh, dh = y.cpu().double().numpy(), do.cpu().double().numpy()
    want, mag = moe_ref.combine(yh, s, w.astype(np.float64))
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= (k + 1) * U * mag + U * np.abs(want))
    prod = np.where(s[:, :, None] >= 0, dh[:, None, :] * yh[s], 0.0)
    n = 8 * -(-cols // 2048) + 12
    assert np.all(np.abs(dw.cpu().double().numpy() - prod.sum(2)) <= n * U * np.abs(prod).sum(2))


def test_a_routing_names_each_row_once():
    x = torch.randn(3000, 40, device=dev())
    x[x < -1.5] = -float("inf")
    r = mx.routing(3000, 40, 6, device=dev())
    mx.mx_route(x, r, token_mask=(torch.rand(3000, device=dev()) > 0.2).to(torch.uint8))
    rows = r.slot_row[r.slot_row >= 0].cpu().numpy()
    assert np.array_equal(np.sort(rows), np.arange(int(r.group_offsets[-1])))
