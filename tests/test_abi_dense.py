"""Refusals of the dense layer's operators and of token scoring: bad arguments are
rejected on the host, before any device work."""
import ctypes
import os

import pytest

NUL, SHAPE, ALIGN, FORMAT, UNSUP = 1, 2, 3, 4, 5
FAKE = 0x100000  # never dereferenced: every call fails its checks or has nothing to do


@pytest.fixture(scope="module")
def mx():
    import microscaling_precision_gemm_amd as mx
    if not os.path.exists(mx.LIB_PATH):
        from microscaling_precision_gemm_amd.build import build
        build()
    mx.load()
    return mx


def weights(mx, fmt=2, layout=0, rows=8, cols=64, codes=FAKE, scales=FAKE, ts=FAKE):
    return ctypes.byref(mx._Tensor(fmt, layout, rows, cols, codes, scales, ts))


def test_linear(mx):
    L = mx.load()

    def call(w, x=FAKE, ldx=64, M=4, out=FAKE, dt=0, ldo=8, **ep):
        e = mx._Epilogue(**ep)
        return L.mx_linear(x, ldx, M, w, ctypes.byref(e), out, dt, ldo, None)

    ok = weights(mx)
    assert call(None) == NUL and call(ok, x=None) == NUL and call(ok, out=None) == NUL
    assert call(weights(mx, codes=None)) == NUL and call(weights(mx, fmt=3, ts=None)) == NUL
    assert call(weights(mx, fmt=9)) == FORMAT and call(ok, dt=2) == FORMAT
    assert call(ok, act=5) == FORMAT and call(ok, act=-1) == FORMAT and call(ok, bias=FAKE, bias_dt=3) == FORMAT
    for fmt in (6, 7):  # FP6
        assert call(weights(mx, fmt=fmt)) == UNSUP
    assert call(weights(mx, layout=1, rows=32, cols=1024), ldx=1024, ldo=32) == UNSUP
    assert call(weights(mx, cols=48)) == SHAPE and call(weights(mx, fmt=3, cols=48)) == SHAPE
    assert call(ok, M=-1) == SHAPE and call(ok, M=1 << 26) == SHAPE and call(ok, ldx=56) == SHAPE
    assert call(ok, ldo=7) == SHAPE and call(weights(mx, rows=1 << 26), ldo=1 << 26) == SHAPE
    assert call(weights(mx, rows=1 << 20), M=1 << 16, ldo=1 << 20) == SHAPE
    assert call(ok, residual=FAKE, ld_residual=7) == SHAPE and call(ok, z=FAKE, ld_z=4) == SHAPE
    assert call(ok, x=FAKE + 8) == ALIGN and call(ok, ldx=68) == ALIGN and call(ok, out=FAKE + 1) == ALIGN
    assert call(ok, bias=FAKE + 1) == ALIGN and call(ok, bias=FAKE + 2, bias_dt=1) == ALIGN
    assert call(ok, residual=FAKE + 1, ld_residual=8) == ALIGN
    assert call(ok, z=FAKE + 2, ld_z=8, dt=1) == ALIGN
    for drop in (-0.1, 1.0, 2.0, float("nan")):
        assert call(ok, drop=drop) == UNSUP
    assert call(ok, M=0, x=None, out=None) == 0
    assert L.mx_linear(FAKE, 64, 0, ok, None, None, 0, 8, None) == 0
    assert call(weights(mx, rows=0, codes=None, scales=None), out=None, ldo=0) == 0


def test_epilogue_backward(mx):
    L, rng = mx.load(), mx._Rng(0, 0)

    def call(do=FAKE, dt=0, rows=4, cols=8, ldd=8, z=FAKE, ldz=8, act=2, drop=0.1, dz=FAKE, lddz=8, db=None, ws=None,
             size=0):
        return L.mx_epilogue_backward(do, dt, rows, cols, ldd, z, ldz, act, drop, rng, dz, lddz, db, ws, size, None)

    assert call(do=None) == NUL and call(z=None) == NUL
    assert call(dt=2) == FORMAT and call(act=5) == FORMAT
    assert call(rows=-1) == SHAPE and call(cols=-1) == SHAPE and call(rows=1 << 31) == SHAPE
    assert call(cols=1 << 31) == SHAPE and call(ldd=7) == SHAPE and call(ldz=7) == SHAPE and call(lddz=7) == SHAPE
    assert call(do=FAKE + 1) == ALIGN and call(z=FAKE + 1) == ALIGN and call(dz=FAKE + 1) == ALIGN
    assert call(db=FAKE + 2) == ALIGN and call(drop=1.0) == UNSUP and call(drop=float("nan")) == UNSUP
    need = mx.mx_epilogue_workspace_bytes(4096, 64)
    assert need > 0 and need % 4 == 0
    big = dict(rows=4096, cols=64, ldd=64, ldz=64, lddz=64, db=FAKE)
    assert call(**big) == NUL and call(**big, ws=FAKE, size=need - 1) == SHAPE
    assert call(**big, ws=FAKE + 8, size=need) == ALIGN
    assert call(rows=0, do=None, z=None, dz=None) == 0 and call(cols=0, ldd=0, ldz=0, lddz=0, do=None, z=None) == 0
    assert call(dz=None) == 0
    for args in ((-1, 8), (8, -1), (1 << 31, 8), (8, 1 << 31), (0, 8), (8, 0), (1, 64)):
        assert mx.mx_epilogue_workspace_bytes(*args) == 0


def test_dropout(mx):
    L, rng = mx.load(), mx._Rng(0, 0)

    def call(x=FAKE, dt=0, rows=4, cols=8, ldx=8, r=None, ldr=0, drop=0.5, out=FAKE, ldo=8):
        return L.mx_dropout(x, dt, rows, cols, ldx, r, ldr, drop, rng, out, ldo, None)

    assert call(x=None) == NUL and call(out=None) == NUL and call(dt=2) == FORMAT
    assert call(rows=-1) == SHAPE and call(cols=-1) == SHAPE and call(rows=1 << 31) == SHAPE
    assert call(ldx=7) == SHAPE and call(ldo=7) == SHAPE and call(r=FAKE, ldr=7) == SHAPE
    assert call(x=FAKE + 1) == ALIGN and call(out=FAKE + 2, dt=1) == ALIGN and call(r=FAKE + 1, ldr=8) == ALIGN
    for drop in (-1e-9, 1.0, float("inf"), float("nan")):
        assert call(drop=drop) == UNSUP
    assert call(rows=0, x=None, out=None) == 0 and call(cols=0, ldx=0, ldo=0, x=None, out=None) == 0


def scoring(mx, tokens=4, vocab=50, topk=2, **kw):
    f = dict.fromkeys(("logp", "entropy", "row_max", "log_sum", "top_id", "top_logp"), FAKE)
    return ctypes.byref(mx._Logprobs(tokens, vocab, topk, **{**f, **kw}))


def test_logprob(mx):
    L = mx.load()

    def call(p, x=FAKE, dt=0, ld=50, target=FAKE, scale=1.0, ws=None, size=0):
        return L.mx_logprob(x, dt, ld, target, scale, p, ws, size, None)

    ok = scoring(mx)
    assert call(None) == NUL and call(ok, x=None) == NUL and call(ok, dt=2) == FORMAT
    for n in ("logp", "entropy", "row_max", "log_sum", "top_id", "top_logp"):
        assert call(scoring(mx, **{n: None})) == NUL
        assert call(scoring(mx, **{n: FAKE + 2})) == ALIGN
    for bad in (dict(tokens=-1), dict(tokens=(1 << 21) + 1), dict(vocab=0), dict(vocab=1 << 31), dict(topk=-1),
                dict(topk=33), dict(vocab=1, topk=2)):
        assert call(scoring(mx, **bad), ld=1 << 32) == SHAPE
    assert call(ok, ld=49) == SHAPE
    assert call(ok, x=FAKE + 1) == ALIGN and call(ok, x=FAKE + 2, dt=1) == ALIGN and call(ok, target=FAKE + 4) == ALIGN
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(ok, scale=scale) == UNSUP
    # few long rows are scored in parts
    need = mx.mx_logprob_workspace_bytes(2, 100000, 5)
    assert need > 0 and need % 8 == 0
    few = scoring(mx, tokens=2, vocab=100000, topk=5)
    assert call(few, ld=100000) == NUL and call(few, ld=100000, ws=FAKE, size=need - 1) == SHAPE
    assert call(few, ld=100000, ws=FAKE + 8, size=need) == ALIGN
    for args in ((0, 100000, 5), (-1, 100000, 5), (2, 0, 0), (2, 1 << 31, 5), (2, 100000, 33), (2, 100000, -1),
                 (5000, 100000, 5), (2, 1000, 5), ((1 << 21) + 1, 100000, 5)):
        assert mx.mx_logprob_workspace_bytes(*args) == 0
    assert call(scoring(mx, tokens=0, **dict.fromkeys(("logp", "entropy", "row_max", "log_sum", "top_id", "top_logp"))),
                x=None) == 0


def test_logprob_backward(mx):
    L = mx.load()

    def call(p, x=FAKE, dt=0, ld=50, target=FAKE, scale=1.0, dl=FAKE, dh=FAKE, dx=FAKE, ldd=50):
        return L.mx_logprob_backward(x, dt, ld, target, scale, p, dl, dh, dx, ldd, None)

    ok = scoring(mx)
    assert call(None) == NUL and call(ok, x=None) == NUL and call(ok, dx=None) == NUL
    for n in ("entropy", "row_max", "log_sum"):
        assert call(scoring(mx, **{n: None})) == NUL
    assert call(ok, ldd=49) == SHAPE and call(ok, ld=49) == SHAPE and call(scoring(mx, topk=40)) == SHAPE
    assert call(ok, dx=FAKE + 1) == ALIGN and call(ok, dl=FAKE + 2) == ALIGN and call(ok, dh=FAKE + 2) == ALIGN
    assert call(ok, scale=0.0) == UNSUP and call(ok, dt=3) == FORMAT
    assert call(scoring(mx, tokens=0), x=None, dx=None) == 0


def test_binding_refuses_mismatched_tensors(mx):
    import torch
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    b = torch.bfloat16
    W = mx.MXTensor(2, 8, 64, z(8, 32, dt=torch.uint8), z(8, 2, dt=torch.uint8))
    s = mx.Logprobs(4, 50, 2, device="cpu")
    i64 = torch.int64
    bad = [
        lambda: mx.mx_linear(z(4, 64), W, z(4, 8)),                               # x must be bf16
        lambda: mx.mx_linear(z(4, 32, dt=b), W, z(4, 8)),
        lambda: mx.mx_linear(z(4, 64, dt=b), W, z(4, 9)),
        lambda: mx.mx_linear(z(64, 4, dt=b).t(), W, z(4, 8)),                     # columns not adjacent
        lambda: mx.mx_linear(z(4, 64, dt=b), W, z(4, 8), bias=z(9)),
        lambda: mx.mx_linear(z(4, 64, dt=b), W, z(4, 8), bias=z(16)[::2]),
        lambda: mx.mx_linear(z(4, 64, dt=b), W, z(4, 8), bias=z(8, dt=i64)),
        lambda: mx.mx_linear(z(4, 64, dt=b), W, z(4, 8), residual=z(4, 8, dt=b)),
        lambda: mx.mx_linear(z(4, 64, dt=b), W, z(4, 8), z=z(3, 8)),
        lambda: mx.mx_epilogue_backward(z(4, 8), None, z(4, 8), act=1),
        lambda: mx.mx_epilogue_backward(z(4, 8), z(4, 8, dt=b), z(4, 8), act=1),
        lambda: mx.mx_epilogue_backward(z(4, 8), z(4, 8), z(4, 7), act=1),
        lambda: mx.mx_epilogue_backward(z(4, 8), z(4, 8), z(4, 8), z(4), act=1),
        lambda: mx.mx_dropout(z(4, 8), z(4, 9), 0.1),
        lambda: mx.mx_dropout(z(4, 8), z(4, 8, dt=b), 0.1),
        lambda: mx.mx_dropout(z(4, 8), z(4, 8), 0.1, residual=z(3, 8)),
        lambda: mx.mx_logprob(z(4, 51), z(4, dt=i64), s),
        lambda: mx.mx_logprob(z(4, 50), z(4, dt=torch.int32), s),
        lambda: mx.mx_logprob(z(4, 50, dt=torch.float16), z(4, dt=i64), s),
        lambda: mx.mx_logprob_backward(z(4, 50), z(4, dt=i64), s, z(5), None, z(4, 50)),
        lambda: mx.mx_logprob_backward(z(4, 50), z(4, dt=i64), s, None, None, z(4, 50, dt=b)),
        lambda: mx.Logprobs(4, 10, 11, device="cpu"),
        lambda: mx.Logprobs(4, 100, 33, device="cpu"),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(mx.MXError):
            f()
    with pytest.raises(AttributeError):
        s.logp = z(4)


def test_tensors_of_another_device(mx, monkeypatch):
    """One tensor elsewhere (host memory, say) is refused, whichever it is."""
    import torch

    class Here(torch.Tensor):
        def get_device(self):
            return 0

    monkeypatch.setattr(mx, "_raw_stream", (lambda device: 0, lambda: 0))
    f32, b, i64, u8 = torch.float32, torch.bfloat16, torch.int64, torch.uint8
    T = lambda *shape, dt=f32: torch.zeros(shape, dtype=dt).as_subclass(Here)
    W = lambda t: mx.MXTensor(mx.FORMATS["nvfp4"], 8, 64, t["codes"], t["scales"], t["ts"])
    s = mx.Logprobs(4, 50, 3, device="cpu")
    s.__dict__["workspace"] = s.workspace.as_subclass(Here)
    calls = [
        (dict(x=T(4, 64, dt=b), codes=T(8, 32, dt=u8), scales=T(8, 4, dt=u8), ts=T(1), bias=T(8), z=T(4, 8),
              residual=T(4, 8), out=T(4, 8)),
         lambda t: mx.mx_linear(t["x"], W(t), t["out"], bias=t["bias"], z=t["z"], residual=t["residual"])),
        (dict(d_out=T(4, 8), z=T(4, 8), d_z=T(4, 8), d_bias=T(8), workspace=T(64, dt=u8)),
         lambda t: mx.mx_epilogue_backward(t["d_out"], t["z"], t["d_z"], t["d_bias"], act=1,
                                           workspace=t["workspace"])),
        (dict(x=T(4, 8), out=T(4, 8), residual=T(4, 8)),
         lambda t: mx.mx_dropout(t["x"], t["out"], 0.1, residual=t["residual"])),
        (dict(x=T(4, 50), target=T(4, dt=i64)), lambda t: mx.mx_logprob(t["x"], t["target"], s)),
        (dict(x=T(4, 50), target=T(4, dt=i64), dl=T(4), dh=T(4), out=T(4, 50)),
         lambda t: mx.mx_logprob_backward(t["x"], t["target"], s, t["dl"], t["dh"], t["out"])),
    ]
    for tensors, call in calls:
        for name in tensors:
            with pytest.raises(mx.MXError, match="current device"):
                call({**tensors, name: tensors[name].as_subclass(torch.Tensor)})
    s.__dict__["workspace"] = s.workspace.as_subclass(torch.Tensor)
    with pytest.raises(mx.MXError, match="current device"):
        calls[3][1](calls[3][0])


def test_packed_structures(mx):
    """The bytes that mx_linear is given are those of the structures."""
    import torch
    e = (3, 1, FAKE, FAKE + 64, 2 ** 40, FAKE + 128, 7, 0.25, 2 ** 64 - 1, 2 ** 63)
    assert mx._PACK_EPILOGUE(*e) == bytes(mx._Epilogue(*e[:8], mx._Rng(*e[8:])))
    W = mx.MXTensor(3, 8, 64, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8), None)
    assert mx._weights(W, -1) == bytes(W.desc())
    W.tensor_scale = torch.ones(1)
    assert mx._weights(W, -1) == bytes(W.desc())
