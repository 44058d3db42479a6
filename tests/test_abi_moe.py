"""Refusals of the operators around the expert products: every bad argument
is turned down on the host with its status, before any device work (there is
no GPU where this runs, so an accepted call would return MX_ERR_HIP)."""
import ctypes
import os

import pytest

FAKE = 0x100000  # 16-byte aligned, never dereferenced
NUL, SHAPE, ALIGN, FORMAT, UNSUP = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def mx():
    import microscaling_precision_gemm_amd as mx
    if not os.path.exists(mx.LIB_PATH):
        from microscaling_precision_gemm_amd.build import build
        build()
    mx.load()
    return mx


def routing(mx, tokens=1000, experts=8, topk=2, **over):
    names = ("expert", "weight", "slot_row", "row_index", "group_offsets", "counts", "valid", "prob_sum", "loss")
    return ctypes.byref(mx._Routing(tokens, experts, topk, *(over.get(n, FAKE) for n in names)))


def test_route(mx):
    L = mx.load()
    need = L.mx_route_workspace_bytes(1000, 8)
    assert need > 0 and L.mx_route_workspace_bytes(64, 8) == 0
    assert L.mx_route_workspace_bytes(-1, 8) == 0 and L.mx_route_workspace_bytes(8, 0) == 0

    def call(r, logits=FAKE, dt=0, ld=8, flags=0, ws=FAKE, wsb=need):
        return L.mx_route(logits, dt, ld, None, flags, r, ws, wsb, None)

    assert call(None) == NUL
    assert call(routing(mx), logits=None) == NUL
    assert call(routing(mx), dt=3) == FORMAT
    assert call(routing(mx), flags=2) == UNSUP
    for bad in (dict(tokens=-1), dict(tokens=(1 << 23) + 1), dict(experts=0), dict(experts=1025), dict(topk=0),
                dict(topk=9), dict(experts=64, topk=17)):
        assert call(routing(mx, **bad), ld=2000) == SHAPE, bad
    assert call(routing(mx), ld=7) == SHAPE
    for n in ("expert", "weight", "slot_row", "row_index", "group_offsets", "counts", "valid", "prob_sum", "loss"):
        assert call(routing(mx, **{n: None})) == NUL, n
        assert call(routing(mx, **{n: FAKE + 2})) == ALIGN, n
    for n in ("group_offsets", "counts", "valid"):
        assert call(routing(mx, **{n: FAKE + 4})) == ALIGN, n
    assert call(routing(mx), logits=FAKE + 1) == ALIGN
    assert call(routing(mx), logits=FAKE + 2, dt=1) == ALIGN
    assert call(routing(mx), ws=None) == NUL
    assert call(routing(mx), wsb=need - 1) == SHAPE
    assert call(routing(mx), ws=FAKE + 8) == ALIGN


def test_route_backward(mx):
    L = mx.load()

    def call(r, logits=FAKE, dt=0, ld=8, flags=0, dw=FAKE, dl=FAKE, dx=FAKE, ldd=8):
        return L.mx_route_backward(logits, dt, ld, None, flags, r, dw, dl, dx, ldd, None)

    assert call(None) == NUL
    assert call(routing(mx), dx=None) == NUL
    assert call(routing(mx), ldd=7) == SHAPE
    assert call(routing(mx), dx=FAKE + 1) == ALIGN
    assert call(routing(mx), dw=FAKE + 2) == ALIGN and call(routing(mx), dl=FAKE + 2) == ALIGN
    assert call(routing(mx), flags=4) == UNSUP
    assert call(routing(mx, topk=9)) == SHAPE
    for n in ("expert", "counts", "valid"):
        assert call(routing(mx, **{n: None})) == NUL
    # nothing to do; what only the forward pass writes may be missing
    free = dict(weight=None, slot_row=None, row_index=None, group_offsets=None, prob_sum=None, loss=None)
    assert call(routing(mx, tokens=0, **free), logits=None, dx=None) == 0


def saved(mx, fmt=1, layout=0, rows=4, cols=128, codes=FAKE, scales=FAKE):
    return ctypes.byref(mx._Tensor(fmt, layout, rows, cols, codes, scales, FAKE))


def test_swiglu(mx):
    L, rng = mx.load(), mx._Rng(0, 0)

    def call(h=FAKE, dt=0, rows=4, cols=64, ldh=128, y=FAKE, ldy=64, s=None, rnd=0, amax=None):
        return L.mx_swiglu(h, dt, rows, cols, ldh, y, ldy, s, rnd, rng, amax, None)

    assert call(h=None) == NUL and call(y=None) == NUL
    assert call(dt=2) == FORMAT and call(rnd=2) == FORMAT
    assert call(cols=48, ldh=128) == SHAPE and call(rows=-1) == SHAPE and call(cols=-32) == SHAPE
    assert call(ldh=120) == SHAPE and call(ldy=56) == SHAPE
    assert call(ldh=132) == ALIGN and call(h=FAKE + 8) == ALIGN and call(y=FAKE + 2) == ALIGN
    assert call(amax=FAKE + 2) == ALIGN
    assert call(s=saved(mx, fmt=9)) == FORMAT
    assert call(s=saved(mx, fmt=2)) == UNSUP and call(s=saved(mx, fmt=3)) == UNSUP
    assert call(s=saved(mx, rows=5)) == SHAPE and call(s=saved(mx, cols=64)) == SHAPE
    assert call(s=saved(mx, codes=None)) == NUL and call(s=saved(mx, scales=FAKE + 4)) == ALIGN
    assert call(rows=32, cols=512, ldh=1024, ldy=512, s=saved(mx, layout=1, rows=32, cols=1024)) == UNSUP
    assert call(rows=0, h=None, y=None) == 0


def test_swiglu_backward(mx):
    L = mx.load()

    def call(s, dy=FAKE, dt=0, rows=4, cols=64, lddy=64, dh=FAKE, lddh=128, ys=None):
        return L.mx_swiglu_backward(s, dy, dt, rows, cols, lddy, dh, lddh, ys, None)

    ok = saved(mx)
    assert call(None) == NUL and call(ok, dy=None) == NUL and call(ok, dh=None) == NUL
    assert call(ok, dt=7) == FORMAT
    assert call(ok, cols=33) == SHAPE and call(ok, lddy=32) == SHAPE and call(ok, lddh=64) == SHAPE
    assert call(saved(mx, rows=3)) == SHAPE and call(saved(mx, fmt=6)) == UNSUP
    assert call(ok, dy=FAKE + 4) == ALIGN and call(ok, lddh=130) == ALIGN
    assert call(ok, ys=saved(mx, cols=128)) == SHAPE and call(ok, ys=saved(mx, fmt=2, cols=64)) == UNSUP
    assert call(saved(mx, rows=0), dy=None, dh=None, rows=0) == 0


def test_wgrad(mx):
    L = mx.load()

    def call(x, dy=FAKE, ld=64, rows=4, n=64, index=None, groups=2, off=FAKE, dw=FAKE, dt=1, ldw=128, flags=0,
             ws=None, size=0):
        return L.mx_wgrad_grouped(dy, ld, rows, n, x, index, groups, off, dw, dt, ldw, flags, ws, size, None)

    ok = saved(mx)
    assert call(None) == NUL and call(ok, dy=None) == NUL and call(ok, dw=None) == NUL
    assert call(ok, off=None) == NUL
    assert call(ok, flags=2) == UNSUP and call(ok, dt=4) == FORMAT
    assert call(ok, groups=0) == SHAPE and call(ok, rows=-1) == SHAPE and call(ok, n=-8) == SHAPE
    assert call(ok, rows=5) == SHAPE and call(ok, ld=56) == SHAPE and call(ok, ldw=96) == SHAPE
    assert call(saved(mx, rows=0), index=FAKE) == SHAPE
    for fmt in (2, 3, 6, 7):
        assert call(saved(mx, fmt=fmt)) == UNSUP
    assert call(saved(mx, layout=1, rows=32, cols=1024), rows=32, ldw=1024) == UNSUP
    assert call(ok, ld=68) == ALIGN and call(ok, dy=FAKE + 2) == ALIGN and call(ok, dw=FAKE + 2) == ALIGN
    assert call(ok, index=FAKE + 2) == ALIGN and call(ok, off=FAKE + 4) == ALIGN
    assert call(ok, n=0, dy=None, dw=None) == 0
    # one tile of dW and many rows: summed in parts
    need = mx.mx_wgrad_workspace_bytes(8192, 64, 128, 1)
    assert need > 0 and need % 4 == 0
    long = dict(x=saved(mx, rows=8192), rows=8192, groups=1, off=None)
    assert call(**long) == NUL and call(**long, ws=FAKE, size=need - 1) == SHAPE
    assert call(**long, ws=FAKE + 8, size=need) == ALIGN
    for args in ((-1, 64, 128, 1), (8192, 0, 128, 1), (8192, 64, 0, 1), (8192, 64, 128, 0), (0, 64, 128, 1),
                 (4096, 4096, 4096, 1), (1 << 31, 64, 128, 1)):
        assert mx.mx_wgrad_workspace_bytes(*args) == 0


def test_combine(mx):
    L = mx.load()

    def fwd(y=FAKE, dt=0, rows=9, cols=64, ld=64, s=FAKE, w=FAKE, t=4, k=2, out=FAKE, odt=0, ldo=64):
        return L.mx_combine(y, dt, rows, cols, ld, s, w, t, k, out, odt, ldo, None)

    assert fwd(y=None) == NUL and fwd(s=None) == NUL and fwd(out=None) == NUL
    assert fwd(dt=2) == FORMAT and fwd(odt=2) == FORMAT
    assert fwd(k=0) == SHAPE and fwd(t=-1) == SHAPE and fwd(rows=-1) == SHAPE and fwd(ld=56) == SHAPE
    assert fwd(ldo=63) == SHAPE
    assert fwd(y=FAKE + 2) == ALIGN and fwd(ld=65) == ALIGN and fwd(s=FAKE + 2) == ALIGN
    assert fwd(w=FAKE + 2) == ALIGN and fwd(out=FAKE + 1) == ALIGN
    assert fwd(t=0, s=None, out=None) == 0

    def bwd(do=FAKE, dt=0, lddo=64, y=FAKE, ldy=64, rows=9, cols=64, s=FAKE, w=FAKE, t=4, k=2, dy=FAKE, lddy=64,
            dw=FAKE):
        return L.mx_combine_backward(do, dt, lddo, y, ldy, rows, cols, s, w, t, k, dy, lddy, dw, None)

    assert bwd(do=None) == NUL and bwd(y=None) == NUL and bwd(s=None) == NUL
    assert bwd(dt=3) == FORMAT
    assert bwd(rows=-1) == SHAPE and bwd(ldy=32) == SHAPE and bwd(lddy=32) == SHAPE and bwd(k=0) == SHAPE
    assert bwd(lddo=66) == ALIGN and bwd(dy=FAKE + 8) == ALIGN and bwd(dw=FAKE + 2) == ALIGN
    assert bwd(dy=None, dw=None, y=None) == 0 and bwd(t=0, do=None, s=None) == 0


def test_binding_refuses_mismatched_tensors(mx):
    import torch
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    X = mx.MXTensor(1, 4, 64, z(4, 64, dt=torch.uint8), z(4, 2, dt=torch.uint8))
    slots, w = z(3, 2, dt=torch.int32), z(3, 2)
    bad = [
        lambda: mx.mx_swiglu(z(4, 64), z(4, 64)),                        # h is not twice as wide
        lambda: mx.mx_swiglu(z(4, 128), z(4, 64, dt=torch.bfloat16)),    # another dtype
        lambda: mx.mx_swiglu(z(128, 4).t(), z(4, 64)),                   # columns not adjacent
        lambda: mx.mx_swiglu_backward(X, z(4, 32), z(3, 64)),
        lambda: mx.mx_wgrad_grouped(z(4, 8), X, None, 1, None, z(8, 64)),  # dY must be bf16
        lambda: mx.mx_wgrad_grouped(z(4, 8, dt=torch.bfloat16), X, None, 2, z(2, dt=torch.int64), z(16, 64)),
        lambda: mx.mx_combine(z(6, 16), slots, z(3, 3), z(3, 16)),
        lambda: mx.mx_combine(z(6, 16), slots.long(), w, z(3, 16)),
        lambda: mx.mx_combine(z(6, 16), slots, w, z(2, 16)),
        lambda: mx.mx_combine_backward(z(3, 16), None, slots, w, z(6, 16), z(3, 2)),
        lambda: mx.mx_combine_backward(z(3, 16), z(6, 16), slots, w, z(5, 16), None),
    ]
    r = mx.Routing(4, 8, 2, device="cpu")
    bad += [
        lambda: mx.mx_route(z(4, 9), r),
        lambda: mx.mx_route(z(4, 8), r, token_mask=z(4)),
        lambda: mx.mx_route_backward(z(4, 8), r, z(4, 3), None, z(4, 8)),
        lambda: mx.mx_route_backward(z(4, 8), r, None, z(2), z(4, 8)),
        lambda: mx.mx_route_backward(z(4, 8), r, None, None, z(4, 8, dt=torch.bfloat16)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(mx.MXError):
            f()
