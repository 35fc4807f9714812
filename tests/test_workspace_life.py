"""How long the binding's cached workspaces live, and what they hold: a CUDA graph keeps the address of the one it
was captured with."""
import gc
import weakref

import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4


@pytest.fixture
def cpu(monkeypatch):
    """No GPU: one stream, handle 7; .capturing says whether it captures."""
    class State:
        capturing = False

    monkeypatch.setattr(w4, "_GEMM_WS", {})
    monkeypatch.setattr(w4, "_GEMM_WS_OLD", {}, raising=False)
    monkeypatch.setattr(w4, "_stream", lambda *a: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: State.capturing)
    return State


def get(need):
    return w4.gemm_workspace(0, 0, 0, "cpu", None, need=need)


def test_a_workspace_that_was_outgrown_is_kept(cpu):
    small = weakref.ref(get(64))
    at = small().data_ptr()
    big = get(4096)
    gc.collect()
    assert small() is not None and small().data_ptr() == at
    assert get(64) is big and get(4096) is big


def test_a_workspace_made_during_capture_is_the_graphs_own(cpu):
    cpu.capturing = True
    a = get(2 << 20)
    assert a.numel() >= 2 << 20 and not bool(a[: 1 << 20].any())
    b = get(2 << 20)
    assert b is not a and w4._GEMM_WS == {}
    cpu.capturing = False
    c = get(64)
    cpu.capturing = True
    assert get(64) is c and get(32) is c  # made before the capture, and large enough: used
    d = get(4096)
    cpu.capturing = False
    assert d is not c and get(64) is c


def test_after_a_timeout_workspaces_are_zero_and_kept(cpu, monkeypatch):
    class TimedOut:
        @staticmethod
        def w4a4_check(stream):
            return 8

        @staticmethod
        def w4a4_last_error():
            return b"a bounded wait gave up"

    small = get(64)
    big = get(4096)
    for t in (small, big):
        t.fill_(1)
    monkeypatch.setattr(w4, "load_library", lambda *a, **k: TimedOut)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_check()
    refs = weakref.ref(small), weakref.ref(big)
    assert not bool(small.any()) and not bool(big.any())
    at = big.data_ptr()
    del small, big
    gc.collect()
    assert all(r() is not None for r in refs)
    assert get(4096).data_ptr() == at  # zero again, so it serves the next call


@pytest.mark.gpu
def test_a_graph_outlives_the_workspace_it_was_captured_with():
    from w4a4_testutil import device

    dev = device()
    M, K, N = 257, 8224, 10100  # the last wave is cut
    gen = torch.Generator(dev).manual_seed(2)
    qw, qa = (w4.mxfp4_rotate_quantize(torch.randn(r, K, device=dev, generator=gen)) for r in (N, M))
    wq = w4.h32_q4_0_pack_weights(torch.randn(5120, 1024, device=dev, generator=gen))
    aq = w4.w4a4_rotate_quantize_act(torch.randn(512, 1024, device=dev, generator=gen))
    need = w4.mxfp4_gemm_workspace_bytes(M, N, K)
    assert 0 < need
    want = w4.mxfp4_gemm(qw, qa, ws=torch.zeros(need, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    key = (torch.device(dev).index, s.cuda_stream)
    w4._GEMM_WS.pop(key, None)
    y = torch.empty_like(want)
    with torch.cuda.stream(s):
        w4.mxfp4_gemm(qw, qa, y=y)  # the workspace of this stream
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            w4.mxfp4_gemm(qw, qa, y=y)
        first = w4._GEMM_WS[key].data_ptr()
        w4.gemm_workspace(0, 0, 0, dev, need=2 * need)  # a product that needs more
        assert w4._GEMM_WS[key].data_ptr() != first
        other = [torch.ones(need, dtype=torch.uint8, device=dev) for _ in range(4)]  # would take the freed block
        torch.cuda.synchronize()
        for _ in range(3):
            y.zero_()
            graph.replay()
            w4.w4a4_gemm(wq, aq)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        assert all(bool((t == 1).all()) for t in other)
    w4.w4a4_check()


@pytest.mark.gpu
@pytest.mark.parametrize("product", ["mxfp4", "int4"])
def test_products_captured_without_a_warm_up(product):
    """Two captures on one stream, and a call outside a graph, none of which finds a workspace: each gives the
    product, in any order of replay."""
    from w4a4_testutil import device

    dev = device()
    gen = torch.Generator(dev).manual_seed(3)
    if product == "mxfp4":
        M, K, N = 257, 8224, 10100
        qw, qa = (w4.mxfp4_rotate_quantize(torch.randn(r, K, device=dev, generator=gen)) for r in (N, M))
        need, call = w4.mxfp4_gemm_workspace_bytes(M, N, K), lambda **k: w4.mxfp4_gemm(qw, qa, **k)  # noqa: E731
    else:
        M, K, N = 300, 1024, 640
        wq = w4.h32_q4_0_pack_weights(torch.randn(N, K, device=dev, generator=gen))
        aq = w4.w4a4_rotate_quantize_act(torch.randn(M, K, device=dev, generator=gen))
        need, call = w4.w4a4_gemm_workspace_bytes(M, N, K), lambda **k: w4.w4a4_gemm(wq, aq, **k)  # noqa: E731
    assert need > 0
    want = call(ws=torch.zeros(need, dtype=torch.uint8, device=dev))
    s = torch.cuda.Stream()
    w4._GEMM_WS.pop((torch.device(dev).index, s.cuda_stream), None)
    torch.cuda.synchronize()
    graphs, ys = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        ys.append(torch.zeros_like(want))
        with torch.cuda.graph(g, stream=s):
            call(y=ys[-1])
            call(y=ys[-1])
        graphs.append(g)
    for i in (1, 0, 1, 0):
        ys[i].zero_()
        torch.cuda.synchronize()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[i], want)
        eager = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(eager, want)
    w4.w4a4_check()
