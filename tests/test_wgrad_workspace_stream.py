"""The weight gradient's own workspace belongs to the stream it is written on.
Taken from another stream's pool it could be a block that queued work of that
stream still reads."""
import contextlib

import pytest
import torch

import microscaling_precision_gemm_amd as mx


class Library:
    """Stands for libmx.so: a workspace is wanted, the call is noted."""

    def __init__(self):
        self.calls = []

    def mx_wgrad_workspace_bytes(self, *args):
        return 4096

    def mx_wgrad_grouped(self, *args):
        self.calls.append(args)
        return 0


class Stream:
    cuda_stream = 1234


@pytest.mark.parametrize("other", [False, True])
def test_allocated_for_the_stream_of_the_call(monkeypatch, other):
    lib, stream = Library(), Stream() if other else None
    current, made, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def allocate(*args, **kw):
        made.append((empty(*args, **kw), current[-1]))
        return made[-1][0]

    monkeypatch.setattr(mx, "load", lambda: lib)
    monkeypatch.setattr(mx, "_stream_of", lambda s: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    X = mx.MXTensor(mx.MX_MXFP8_E4M3, 4, 64, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    dW = torch.zeros(8, 64)
    mx.mx_wgrad_grouped(torch.zeros(4, 8, dtype=torch.bfloat16), X, None, 1, None, dW, stream=stream)
    (workspace, owner), = made
    assert owner is stream and current == [None]
    (call,) = lib.calls
    assert call[-3:] == (workspace.data_ptr(), 4096, 1234 if other else 0)


@pytest.mark.gpu
def test_pools_on_the_device():
    dev = torch.device("cuda:0")
    rows, N, K = 8192, 64, 128
    size = mx.mx_wgrad_workspace_bytes(rows, N, K, 1)
    assert size > 0
    X = mx.empty(mx.MX_MXFP8_E4M3, rows, K, dev)
    mx.mx_quantize(torch.randn(rows, K, device=dev), X)
    dy = torch.randn(rows, N, device=dev).to(torch.bfloat16)
    want, got = torch.empty(N, K, device=dev), torch.empty(N, K, device=dev)
    mx.mx_wgrad_grouped(dy, X, None, 1, None, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    # a block of the workspace's size that the current stream still reads when it is freed
    a = torch.full((size // 4,), 3.0, device=dev)
    sums = [a.mul(1.0) for _ in range(20)]
    del a
    mx.mx_wgrad_grouped(dy, X, None, 1, None, got, stream=s)
    torch.cuda.synchronize()
    assert all(bool((t == 3.0).all()) for t in sums)
    assert torch.equal(got, want)
    assert any(seg["stream"] == s.cuda_stream for seg in torch.cuda.memory_snapshot())
