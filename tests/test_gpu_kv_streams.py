"""Attention's workspaces: each stream its own, whatever its handle."""
import ctypes
import threading

import pytest
import torch

import bit_quantized_gemm_qmm_b200 as q
from test_gpu_kv import BF, attention_case, filled_cache, gen, ints, page_tables

pytestmark = pytest.mark.gpu

PER_THREAD = 2  # cudaStreamPerThread: one handle, a stream for each host thread


def finish():
    """Waits for the calling thread's default stream.  A thread that ends with work pending there can leave the
    driver spinning for ever (580.159; seen with the GPU idle)."""
    assert ctypes.CDLL("libcuda.so.1").cuStreamSynchronize(ctypes.c_void_p(PER_THREAD)) == 0


def call(c, x, table, lens, cu, out, lse, stream):
    """qmm_kv_attention through the C ABI on any stream handle (the call itself runs without the interpreter's lock)."""
    T, H, D = x.shape
    s = q.SeqsDesc(table.data_ptr(), cu.data_ptr(), table.shape[0], table.stride(0), table.shape[1])
    st = q.lib().qmm_kv_attention(ctypes.byref(c._desc), x.data_ptr(), H * D, D, out.data_ptr(), H * D, D, lse.data_ptr(),
                                  ctypes.byref(s), lens.data_ptr(), T, H, D ** -0.5, 0, None,
                                  q.QMM_BF16 if x.dtype == BF else q.QMM_F16, stream)
    assert st == q.QMM_OK


def long_case(seed, new):
    """Few items over many positions: every block shares one."""
    n = 9000 + 1000 * seed
    c = filled_cache(n // 64 + 2, 64, 2, 128, 64, seed)
    table = page_tables([n], 64, c.pages, seed)
    x = torch.randn((new, 8, 128), device="cuda", generator=gen(seed)).to(BF)
    return c, x, table, ints([n]), ints([0, new])


@pytest.mark.parametrize("new", [1, 20])
def test_threads_on_their_own_default_streams(new):
    cases = [long_case(s, new) for s in range(4)]
    want = [q.kv_attention(*c) for c in cases]
    outs = [[(torch.full_like(o, 7), torch.full_like(l, 7)) for _ in range(8)] for o, l in want]
    torch.cuda.synchronize()
    start = threading.Barrier(len(cases))
    failed = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            start.wait(60)
            for turn in range(400):
                call(*cases[i], *outs[i][turn % 8], PER_THREAD)
            finish()
        except Exception as e:  # noqa: BLE001 - told to the main thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for (o, l), mine in zip(want, outs):
        for o2, l2 in mine:
            assert torch.equal(o, o2) and torch.equal(l, l2)
    assert q.device_errors() == 0


def test_streams_that_come_and_go():
    """Streams destroyed with work pending, whose handles may come back; their workspaces do not pile up."""
    cu = ctypes.CDLL("libcuda.so.1")
    case = long_case(1, 1)
    want, wl = q.kv_attention(*case)
    outs = [(torch.full_like(want, 7), torch.full_like(wl, 7)) for _ in range(60)]
    torch.cuda.synchronize()
    used = []
    for turn, (o, l) in enumerate(outs):
        s = ctypes.c_void_p()
        assert cu.cuStreamCreate(ctypes.byref(s), 1) == 0  # non-blocking
        call(*case, o, l, s)
        assert cu.cuStreamDestroy_v2(s) == 0
        if turn % 20 == 19:
            torch.cuda.synchronize()
            used.append(torch.cuda.mem_get_info()[0])
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, wl)
    assert used[0] - used[-1] < 100 << 20  # 40 streams' workspaces are 160 MB at least


def test_graphs_and_eager_calls_of_one_stream():
    c, x, table, lens, cu, scale, _, _ = attention_case("long")
    want, wl = q.kv_attention(c, x, table, lens, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        q.kv_attention(c, x, table, lens, cu, out=out, lse=lse)
    with torch.cuda.stream(side):
        for _ in range(20):
            g.replay()
            o2, l2 = q.kv_attention(c, x, table, lens, cu)
    torch.cuda.synchronize()
    for o, l in ((out, lse), (o2, l2)):
        assert torch.equal(o, want) and torch.equal(l, wl)


def test_eager_calls_of_another_thread_while_one_captures():
    """The capture's rules are global by default: what another thread's call asks for must not end it."""
    case, other = long_case(1, 1), long_case(2, 20)
    want, other_want = q.kv_attention(*case), q.kv_attention(*other)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    got, failed = [torch.empty_like(t) for t in other_want], []
    called, captured = threading.Event(), threading.Event()
    torch.cuda.synchronize()

    def eager():
        try:
            torch.cuda.set_device(0)
            for _ in range(5):
                call(*other, *got, PER_THREAD)  # the first of them allocates
            called.set()
            assert captured.wait(60)
            finish()
        except Exception as e:  # noqa: BLE001 - told to the main thread
            failed.append(e)
            called.set()

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.kv_attention(*case, out=out, lse=lse)
        t = threading.Thread(target=eager)
        t.start()
        assert called.wait(60)
        q.kv_attention(*case, out=out, lse=lse)
    captured.set()
    t.join()
    assert not failed
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(got[0], other_want[0]) and torch.equal(got[1], other_want[1])


@pytest.mark.parametrize("op", ["attention", "qmm"])
def test_workspaces_of_graphs_that_are_gone(op):
    """Graphs captured, replayed and dropped, a last replay in flight: right to the end, and their memory comes back."""
    if op == "attention":
        case = long_case(1, 1)
        want = q.kv_attention(*case)
        call_one = lambda out: q.kv_attention(*case, out=out[0], lse=out[1])  # noqa: E731
    else:
        w = q.QuantizedWeight.from_dense(torch.randn((32000, 1024), device="cuda", generator=gen(1)).half(), 4, 64)
        x = torch.randn((1, 1024), device="cuda", generator=gen(2)).half()
        want = (w(x),)
        call_one = lambda out: w(x, out=out[0])  # noqa: E731
    outs = [[torch.full_like(t, 7) for t in want] for _ in range(60)]
    torch.cuda.synchronize()
    free, kept = [], []
    for turn, out in enumerate(outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call_one(out)
        for _ in range(20):
            g.replay()
        if turn % 20 == 7:
            kept.append(g)
        del g
        if turn % 20 == 19:
            free.append(torch.cuda.mem_get_info()[0])
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert free[0] - free[-1] < 60 << 20  # 40 captures' workspaces are 160 MB at least
    for out in outs:
        for t in out:
            t.fill_(7)
    for g in kept:
        g.replay()
    torch.cuda.synchronize()
    for turn, out in enumerate(outs):
        if turn % 20 == 7:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_workspaces_of_threads_that_are_gone():
    """Threads come, call on their default streams, wait and end: their workspaces do not pile up."""
    case = long_case(1, 1)
    want, wl = q.kv_attention(*case)
    outs = [(torch.full_like(want, 7), torch.full_like(wl, 7)) for _ in range(60)]
    torch.cuda.synchronize()
    free, failed = [], []

    def work(o, l):
        try:
            torch.cuda.set_device(0)
            for _ in range(3):
                call(*case, o, l, PER_THREAD)
            finish()
        except Exception as e:  # noqa: BLE001 - told to the main thread
            failed.append(e)

    for turn, (o, l) in enumerate(outs):
        t = threading.Thread(target=work, args=(o, l))
        t.start()
        t.join()
        if turn % 20 == 19:
            free.append(torch.cuda.mem_get_info()[0])
    torch.cuda.synchronize()
    assert not failed
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, wl)
    assert free[0] - free[-1] < 60 << 20  # 40 threads' workspaces are 160 MB at least
