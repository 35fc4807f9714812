"""A caller's `out` of the wrong kind, shape or device is refused before the library is called: needs no GPU
(the library is played by a recorder, and the checks of the inputs' device are off)."""
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4

MAKE = {"Act4": w4.alloc_act4, "Act8": w4.alloc_act8, "Act16": w4.alloc_act16, "MxFp4": w4.alloc_mxfp4,
        "Q4_0Weights": w4.alloc_q4_0}
X = torch.zeros(4, 64)
U8 = torch.zeros(4, 32, dtype=torch.uint8)
EXACT = {  # out holds exactly the result
    "MxFp4": [lambda o: w4.mxfp4_rotate_quantize(X, out=o), lambda o: w4.mxfp4_rmsnorm_quantize(X, out=o),
              lambda o: w4.mxfp4_swiglu_quantize(X, X, out=o),
              lambda o: w4.mxfp4_import(U8, torch.zeros(4, 2, dtype=torch.uint8), out=o)],
    "Act8": [lambda o: w4.w4a8_rmsnorm_quantize_act(X, out=o), lambda o: w4.w4a8_swiglu_quantize_act(X, X, out=o)],
    "Act4": [lambda o: w4.w4a4_rmsnorm_quantize_act(X, out=o), lambda o: w4.w4a4_swiglu_quantize_act(X, X, out=o)],
}
ROOM = {  # out may hold more rows
    "Act4": [lambda o: w4.w4a4_rotate_quantize_act(X, out=o)],
    "Act8": [lambda o: w4.w4a8_rotate_quantize_act(X, out=o)],
    "Act16": [lambda o: w4.w4a16_rotate_act(X, out=o)],
    "Q4_0Weights": [lambda o: w4.h32_q4_0_pack_weights(X, out=o),
                    lambda o: w4.h32_q4_0_pack_weights_imatrix(X, None, out=o),
                    lambda o: w4.q4_0_import(torch.zeros(4 * 2 * 18, dtype=torch.uint8), 64, out=o)],
}
CALLS = [(k, c, exact) for t, exact in ((EXACT, True), (ROOM, False)) for k, cs in t.items() for c in cs]


class _Recorder:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    w4.load_library(build_if_missing=True)
    outs = {k: {"good": f(4, 64, "cpu"), "more": f(9, 64, "cpu"), "fewer": f(3, 64, "cpu"), "wide": f(4, 96, "cpu"),
                "narrow": f(8, 32, "cpu"), "elsewhere": f(4, 64, "meta")} for k, f in MAKE.items()}
    r = _Recorder()
    r.outs = outs
    monkeypatch.setattr(w4, "load_library", lambda *a, **k: r)
    monkeypatch.setattr(w4, "_cuda", lambda *a: None)
    monkeypatch.setattr(w4, "_rows", lambda t, *a: t.shape[1])
    monkeypatch.setattr(w4, "_stream", lambda *a: 0)
    return r


@pytest.mark.parametrize("kind,call,exact", CALLS)
def test_out_is_checked(lib, kind, call, exact):
    for other, outs in lib.outs.items():
        if other != kind:
            with pytest.raises(ValueError, match="out"):
                call(outs["good"])
    for shape in ("fewer", "wide", "narrow", "elsewhere") + (("more",) if exact else ()):
        with pytest.raises(ValueError, match="out"):
            call(lib.outs[kind][shape])
    assert lib.calls == 0
    assert call(lib.outs[kind]["good"]) is lib.outs[kind]["good"]
    if not exact:
        call(lib.outs[kind]["more"])
        assert lib.outs[kind]["more"].rows == 9
    assert lib.calls == (1 if exact else 2)


READ = {"MxFp4": [lambda a: w4.mxfp4_dequantize(a), lambda a: w4.mxfp4_gemm(a, a)],
        "Act4": [lambda a: w4.w4a4_dequantize_act(a)], "Act8": [lambda a: w4.w4a8_dequantize_act(a)]}


@pytest.mark.parametrize("kind,call", [(k, c) for k, cs in READ.items() for c in cs])
def test_operands_read_are_checked(lib, kind, call):
    """An operand of another kind, or one that is not on a GPU, never reaches the library."""
    for other, outs in lib.outs.items():
        with pytest.raises(ValueError):
            call(outs["good"])
    assert lib.calls == 0
