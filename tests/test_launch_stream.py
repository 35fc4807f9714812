"""What a call allocates, it allocates (and fills) on the stream it launches on, also where that is not the
current one."""
import contextlib

import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4


class _Stream:
    def __init__(self, handle, *a, **k):
        self.cuda_stream = handle


class _Recorder:
    """Stands in for libw4a4.so: every call succeeds; sizes are what they would be, or a fixed need."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return getattr(self.lib, name) if name.endswith("_bytes") else (lambda *a: 0)


@pytest.fixture
def streams(monkeypatch):
    """The current stream is 0; .made: the stream and the tensor of each allocation; .read: (tensor, stream) recorded."""
    lib = w4.load_library(build_if_missing=True)
    here = [_Stream(0)]

    class Log:
        made, read = [], []

    @contextlib.contextmanager
    def under(s):
        here.append(s)
        yield
        here.pop()

    def noted(make):
        def f(*a, **k):
            Log.made.append((here[-1].cuda_stream, make(*a, **k)))
            return Log.made[-1][1]
        return f

    monkeypatch.setattr(w4, "load_library", lambda *a, **k: _Recorder(lib))
    monkeypatch.setattr(w4, "_cuda", lambda *a: None)
    monkeypatch.setattr(w4, "_rows", lambda t, *a: t.shape[1])
    monkeypatch.setattr(w4, "_GEMM_WS", {})
    monkeypatch.setattr(w4.MxFp4, "_gpu", property(lambda q: True, lambda q, v: None))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: _Stream(0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: here[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: Log.read.append((t.untyped_storage().data_ptr(),
                                                                                     s.cuda_stream)))
    monkeypatch.setattr(torch, "empty", noted(torch.empty))
    monkeypatch.setattr(torch, "zeros", noted(torch.zeros))
    Log.made, Log.read = [], []
    return Log


X, U8 = torch.zeros(200, 64), torch.zeros(200, 32, dtype=torch.uint8)
IDS = torch.zeros(200, 2, dtype=torch.int32)
CALLS = {
    "h32_q4_0_pack_weights": lambda o, s: w4.h32_q4_0_pack_weights(X, stream=s, expanded=True),
    "h32_q4_0_pack_weights_imatrix": lambda o, s: w4.h32_q4_0_pack_weights_imatrix(X, None, stream=s),
    "q4_0_import": lambda o, s: w4.q4_0_import(torch.zeros_like(U8[:, :36].reshape(-1)[: 36 * 100]), 64, stream=s),
    "w4a4_rotate_quantize_act": lambda o, s: w4.w4a4_rotate_quantize_act(X, stream=s),
    "w4a8_rotate_quantize_act": lambda o, s: w4.w4a8_rotate_quantize_act(X, stream=s),
    "w4a16_rotate_act": lambda o, s: w4.w4a16_rotate_act(X, stream=s),
    "mxfp4_rotate_quantize": lambda o, s: w4.mxfp4_rotate_quantize(X, stream=s),
    "mxfp4_import": lambda o, s: w4.mxfp4_import(U8, U8[:, :2].contiguous(), stream=s),
    "w4a4_rmsnorm_quantize_act": lambda o, s: w4.w4a4_rmsnorm_quantize_act(X, stream=s),
    "w4a8_swiglu_quantize_act": lambda o, s: w4.w4a8_swiglu_quantize_act(X, X, stream=s),
    "mxfp4_rmsnorm_quantize": lambda o, s: w4.mxfp4_rmsnorm_quantize(X, stream=s),
    "w4a4_gemm": lambda o, s: w4.w4a4_gemm(o["w"], o["a4"], stream=s),
    "w4a4_gemm_small_m": lambda o, s: w4.w4a4_gemm_small_m(o["w"], o["a4"], stream=s),
    "w4a4_gemm_partials": lambda o, s: w4.w4a4_gemm_partials(o["w"], o["a4"], stream=s),
    "w4a4_gemm_id": lambda o, s: w4.w4a4_gemm_id(o["w"], 2, o["a4"], IDS, 2, False, stream=s),
    "w4a8_gemm": lambda o, s: w4.w4a8_gemm(o["w"], o["a8"], stream=s),
    "w4a8_gemm_partials": lambda o, s: w4.w4a8_gemm_partials(o["w"], o["a8"], stream=s),
    "w4a16_gemm": lambda o, s: w4.w4a16_gemm(o["w"], o["a16"], stream=s),
    "mxfp4_gemm": lambda o, s: w4.mxfp4_gemm(o["mw"], o["ma"], stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_allocations_are_made_on_the_launch_stream(streams, name):
    o = {"w": w4.alloc_q4_0(100, 64, "cpu"), "a4": w4.alloc_act4(200, 64, "cpu"), "a8": w4.alloc_act8(200, 64, "cpu"),
         "a16": w4.alloc_act16(200, 64, "cpu"), "mw": w4.alloc_mxfp4(100, 64, "cpu"),
         "ma": w4.alloc_mxfp4(200, 64, "cpu")}
    for stream, want in ((None, 0), (0, 0), (_Stream(7), 7), (9, 9)):
        streams.made, streams.read = [], []
        out = CALLS[name](o, stream)
        assert streams.made and {s for s, _ in streams.made} == {want}
        got = out if isinstance(out, torch.Tensor) else out.codes if hasattr(out, "codes") else out.values
        at = got.untyped_storage().data_ptr()
        # the result is read on the current stream next: its memory waits for that before it is used again
        assert ((at, 0) in streams.read) == (want != 0)


def test_a_workspace_is_one_streams(streams):
    a = w4.gemm_workspace(0, 0, 0, "cpu", _Stream(7), need=64)
    assert w4.gemm_workspace(0, 0, 0, "cpu", 7, need=32) is a and [s for s, _ in streams.made] == [7]
    assert w4.gemm_workspace(0, 0, 0, "cpu", None, need=64) is not a and [s for s, _ in streams.made] == [7, 0]


@pytest.mark.gpu
def test_workspace_filled_behind_a_busy_stream():
    """A product on a stream of its own whose workspace is new, while the current stream is busy and the memory
    that a fill on it would have taken holds ones."""
    from w4a4_testutil import device

    dev = device()
    M, K, N = 257, 8224, 10100  # its last wave is cut: the workspace's flags decide what is added
    need = w4.mxfp4_gemm_workspace_bytes(M, N, K)
    assert need > 0
    gen = torch.Generator(dev).manual_seed(1)
    qw, qa = (w4.mxfp4_rotate_quantize(torch.randn(r, K, device=dev, generator=gen)) for r in (N, M))
    want = w4.mxfp4_gemm(qw, qa, ws=torch.zeros(need, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    for _ in range(3):
        s = torch.cuda.Stream()
        w4._GEMM_WS.pop((dev.index, s.cuda_stream), None)
        dirty = torch.ones(need, dtype=torch.uint8, device=dev)
        torch.cuda.synchronize()
        del dirty
        torch.cuda._sleep(20_000_000)  # about 10 ms
        y = w4.mxfp4_gemm(qw, qa, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    w4.w4a4_check()
