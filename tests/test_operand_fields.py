"""The fields of Act8 and MxFp4 operands and what a call is told of them agree, whatever a
program does to the fields: needs no GPU (the library is played by a recorder)."""
import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from hadamard_rotated_w4a4_gb300 import _Act4Desc


class _Recorder:
    """Stands in for libw4a4.so: stamps the descriptors that quantisers get, as the library does, and notes the
    rows of those that the products get."""

    def __init__(self):
        self.rows = []

    @staticmethod
    def _at(d):
        return _Act4Desc.from_address(d) if isinstance(d, int) else d._obj

    def w4a8_rotate_quantize_act(self, x, M, K, ldx, rotate, d, stream):
        d = self._at(d)
        d.rows, d.K, d.tag = M, K, w4.TAG_ACT8 | rotate
        return 0

    def w4a8_gemm_partials(self, w, a, P, stream):
        self.rows.append(self._at(a).rows)
        return 0


@pytest.fixture
def lib(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(w4, "load_library", lambda *a, **k: r)
    monkeypatch.setattr(w4, "_cuda", lambda *a: None)
    monkeypatch.setattr(w4, "_stream", lambda *a: 0)
    return r


def weights(N, K):
    u = torch.zeros(N * K, dtype=torch.uint8)
    return w4.Q4_0Weights(u[: N * K // 2].view(N, K // 2), u, u, N, K, True)


def test_act8_first_rows(lib):
    a = w4.alloc_act8(5, 64, "cpu")
    a.rows = 2
    assert a.desc().rows == 2 and a.scales.shape == (2, 2)
    assert w4.w4a8_gemm_partials(weights(3, 64), a).shape == (2, 3, 2) and lib.rows == [2]
    b = dataclasses.replace(a, rows=1)
    assert (b.rows, b.K, b.rotated, a.rows) == (1, 64, True, 2)
    assert b.desc().rows == 1 and b.desc().codes == a.desc().codes and b.desc().scales == a.desc().scales


def test_act8_larger_out_keeps_its_rows(lib):
    a = w4.alloc_act8(4, 64, "cpu")
    w4.w4a8_rotate_quantize_act(torch.zeros(1, 64), rotate=False, out=a)
    assert a.rows == 4 and not a.rotated
    assert w4.w4a8_gemm_partials(weights(3, 64), a).shape == (4, 3, 2) and lib.rows == [4]


def test_act8_rows_it_does_not_hold(lib):
    for a in (w4.alloc_act8(4, 64, "cpu"), w4.Act8(torch.zeros(4, 64, dtype=torch.int8),
                                                   torch.zeros(32, dtype=torch.uint8), 4, 64, True)):
        a.rows = 5
        with pytest.raises(ValueError):
            a.desc()
        with pytest.raises(ValueError):
            w4.w4a8_gemm_partials(weights(3, 64), a)
    assert lib.rows == []


def test_act8_assigned_buffers():
    a = w4.alloc_act8(4, 64, "cpu")
    codes, scales = torch.ones(4, 64, dtype=torch.int8), torch.zeros(32, dtype=torch.uint8)
    kept = a.scales_buf.data_ptr()
    a.codes = codes
    assert (a.desc().codes, a.desc().scales) == (codes.data_ptr(), kept)
    a.scales_buf = scales
    assert (a.desc().codes, a.desc().scales) == (codes.data_ptr(), scales.data_ptr())
    b = w4.alloc_act8(4, 64, "cpu")
    b.scales_buf = scales
    assert b.desc().scales == scales.data_ptr() and b.desc().codes == b.codes.data_ptr()


def buffers(q):
    return (q.codes, q.scales_buf)


@pytest.mark.parametrize("make", [w4.alloc_act8, w4.alloc_mxfp4])
@pytest.mark.parametrize("how", [copy.deepcopy, lambda q: pickle.loads(pickle.dumps(q)), copy.copy])
@pytest.mark.parametrize("seen", [False, True])
def test_copies(make, how, seen):
    q = make(3, 96, "cpu")
    if seen:  # the views of the buffers exist
        for t in buffers(q):
            t.view(torch.uint8).random_(0, 256)
    q.rotated = False
    p = how(q)
    assert type(p) is type(q) and (p.rows, p.K, p.rotated) == (3, 96, False)
    d, e = q.desc(), p.desc()
    assert (e.rows, e.K, e.tag) == (3, 96, d.tag) and not d.tag & w4.TAG_ROTATED
    assert (e.codes, e.scales) == tuple(t.data_ptr() for t in buffers(p))
    if how is copy.copy:
        assert e.codes == d.codes
    else:
        assert e.codes != d.codes
        p.codes.zero_()
    if seen:
        for a, b in zip(buffers(p)[1:] if how is not copy.copy else buffers(p),
                        buffers(q)[1:] if how is not copy.copy else buffers(q)):
            assert torch.equal(a, b)
    p.rotated = True
    assert p.desc().tag & w4.TAG_ROTATED and not q.desc().tag & w4.TAG_ROTATED


def test_mxfp4_shape_is_fixed():
    """Its scale tiles follow from its rows and K, so neither can be changed."""
    q = w4.alloc_mxfp4(130, 160, "cpu")
    for name, value in (("rows", 1), ("K", 32), ("buf", torch.zeros(4, dtype=torch.uint8))):
        with pytest.raises(AttributeError):
            setattr(q, name, value)
    d = q.desc()
    d.rows = 1000  # a copy
    assert (q.rows, q.K, q.desc().rows) == (130, 160, 130) and ctypes.addressof(d) != ctypes.addressof(q.desc())
    assert q.desc().scales == q.scales_buf.data_ptr()


def test_mxfp4_takes_no_buffer_of_another_size():
    buf = w4.alloc_mxfp4(130, 160, "cpu").buf
    assert w4.MxFp4(130, 160, "cpu", buf=buf).buf is buf
    for other in (buf[:-16], buf.view(torch.int8), torch.zeros(2 * len(buf), dtype=torch.uint8)[::2], buf.view(2, -1)):
        with pytest.raises(ValueError):
            w4.MxFp4(130, 160, "cpu", buf=other)


# ----------------------------------------------------------------- the same on the GPU
@pytest.fixture(scope="module")
def dev():
    from w4a4_testutil import device
    return device()


@pytest.mark.gpu
def test_products_follow_the_fields(dev):
    gen = torch.Generator(dev).manual_seed(0)
    x, w = torch.randn(6, 256, device=dev, generator=gen), torch.randn(40, 256, device=dev, generator=gen)
    wq, a = w4.h32_q4_0_pack_weights(w), w4.w4a8_rotate_quantize_act(x)
    want = w4.w4a8_gemm(wq, a)
    assert torch.equal(w4.w4a8_gemm(wq, dataclasses.replace(a, rows=2)), want[:2])
    assert torch.equal(w4.w4a8_gemm(wq, copy.deepcopy(a)), want)
    # fewer rows into it: the first two are new, the others stay
    w4.w4a8_rotate_quantize_act(x[4:].contiguous(), out=a)
    assert torch.equal(w4.w4a8_gemm(wq, a), torch.cat((want[4:], want[2:])))
    a.rows = 2
    assert torch.equal(w4.w4a8_gemm(wq, a), want[4:])
    mw, ma = w4.mxfp4_rotate_quantize(w), w4.mxfp4_rotate_quantize(x)
    want = w4.mxfp4_gemm(mw, ma)
    for how in (copy.deepcopy, lambda q: pickle.loads(pickle.dumps(q))):
        assert torch.equal(w4.mxfp4_gemm(how(mw), how(ma)), want)
    w4.w4a4_check()
