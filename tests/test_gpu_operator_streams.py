"""Scratch memory of the training-step operators: calls on different streams
never share it, whatever the streams' handles."""
import ctypes
import threading

import pytest
import torch

import ring_allreduce_compressed_gb300 as rra

pytestmark = pytest.mark.gpu

PER_THREAD = 2  # cudaStreamPerThread


class Handle:
    """A stream as the binding takes it, by its handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


def problem(seed, n, vocab, dim):
    """Tokens and gradients of small whole numbers: sums in any order are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    d = torch.randint(-8, 9, (n, dim), generator=g, device="cuda").float()
    want = torch.zeros(vocab, dim, device="cuda").index_add_(0, t, d)
    return t, d, want


def test_per_thread_default_streams_keep_their_scratch_apart():
    """One handle names another stream in every thread.  Two threads' gradients
    of different sizes run at the same time, over and over."""
    problems = [problem(1, 40_000, 3000, 64), problem(2, 9000, 500, 200)]
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(problems))

    def work(k):
        try:
            t, d, want = problems[k]
            dw = [torch.empty_like(want) for _ in range(60)]
            norm = [torch.empty(1, device="cuda") for _ in dw]
            torch.cuda.synchronize()
            start.wait()
            for o, n in zip(dw, norm):
                rra.embedding_grad(d, t, o, stream=Handle(PER_THREAD))
                rra.grad_norm([d], n, norm_type=1, stream=Handle(PER_THREAD))
            torch.cuda.synchronize()
            size = float(d.double().abs().sum())
            for o, n in zip(dw, norm):
                assert torch.equal(o, want)
                assert float(n) == size  # whole numbers below 2^24
        except BaseException as e:  # noqa: BLE001 (reported by the test's own thread)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(problems))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed


def test_threads_that_come_and_go_leave_their_scratch_to_others():
    t, d, want = problem(3, 50_000, 100, 512)
    before, failed = None, []

    def work():
        try:
            dw = torch.empty_like(want)
            torch.cuda.synchronize()
            rra.embedding_grad(d, t, dw, stream=Handle(PER_THREAD))
            torch.cuda.synchronize()
            assert torch.equal(dw, want)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)
    for k in range(30):
        th = threading.Thread(target=work)
        th.start()
        th.join()
        assert not failed, failed
        if k == 4:
            before = torch.cuda.mem_get_info()[0]
    # a call's scratch has more than 6 MB of partial sums; 25 calls since
    assert before - torch.cuda.mem_get_info()[0] < 64_000_000


def test_sparse_codec_on_per_thread_default_streams():
    """Two threads encode and decode messages of different sizes at the same time."""
    failed, start = [], threading.Barrier(2)

    def work(k):
        try:
            n = (3_000_001, 700_003)[k]
            g = torch.Generator(device="cuda").manual_seed(k)
            x = torch.randn(n, generator=g, device="cuda")
            x = torch.where(torch.rand(n, generator=g, device="cuda") < 0.8, torch.zeros_like(x), x)
            back = [torch.empty_like(x) for _ in range(20)]
            hdr = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in back]
            vals, idx = torch.empty_like(x), torch.empty(n, dtype=torch.int32, device="cuda")
            torch.cuda.synchronize()
            start.wait()
            for h, b in zip(hdr, back):
                rra.sparse_encode(x, 0.5, h, vals, idx, stream=Handle(PER_THREAD))
                rra.sparse_decode(h, vals, idx, n, b, stream=Handle(PER_THREAD))
            torch.cuda.synchronize()
            nnz = int((x != 0).sum())
            for h, b in zip(hdr, back):
                assert h.tolist() == [1, nnz]
                assert torch.equal(b, x)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed


def test_sparse_codec_in_a_graph():
    """A stream that is captured keeps the scratch of its calls before."""
    n = 500_003
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, generator=g, device="cuda")
    x = torch.where(torch.rand(n, generator=g, device="cuda") < 0.7, torch.zeros_like(x), x)
    hdr, back = torch.empty(2, dtype=torch.int32, device="cuda"), torch.zeros_like(x)
    vals, idx = torch.empty_like(x), torch.empty(n, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    rra.sparse_encode(x, 0.5, hdr, vals, idx, stream=st)
    rra.sparse_decode(hdr, vals, idx, n, back, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        rra.sparse_encode(x, 0.5, hdr, vals, idx)
        rra.sparse_decode(hdr, vals, idx, n, back)
    for _ in range(2):
        x.copy_(x.flip(0))
        back.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, x)


def new_stream():
    """A stream that no other test has used, and the function that destroys it."""
    rt = torch.cuda.cudart()
    handle = ctypes.c_void_p()
    assert int(rt.cudaStreamCreate(ctypes.addressof(handle))) == 0
    return torch.cuda.ExternalStream(handle.value), lambda: rt.cudaStreamDestroy(handle.value)


def sparse(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, generator=g, device="cuda")
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.7, torch.zeros_like(x), x)


def test_sparse_codec_keeps_a_graph_s_scratch_when_it_grows():
    """A larger call behind the capture takes a buffer of its own."""
    small, large = 300_007, 80_000_003
    x, big = sparse(small, 6), sparse(large, 7)
    hdr, back = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(big)
    vals, idx = torch.empty_like(big), torch.empty(large, dtype=torch.int32, device="cuda")
    st, destroy = new_stream()

    def call(v):
        rra.sparse_encode(v, 0.5, hdr, vals, idx, stream=st)
        rra.sparse_decode(hdr, vals, idx, v.numel(), back, stream=st)
    torch.cuda.synchronize()
    call(x)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call(x)
    call(big)
    st.synchronize()
    assert torch.equal(back, big)
    for seed in (8, 9):
        x.copy_(sparse(small, seed))
        call(big)
        st.synchronize()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back[:small], x) and torch.equal(back[small:], big[small:])
    destroy()


def test_sparse_codec_that_would_grow_in_a_capture_is_refused():
    """The capture stays usable, and so does the stream's scratch."""
    x = sparse(80_000_003, 7)
    hdr, back = torch.empty(2, dtype=torch.int32, device="cuda"), torch.zeros_like(x)
    vals, idx = torch.empty_like(x), torch.empty(x.numel(), dtype=torch.int32, device="cuda")
    y = torch.zeros(4, device="cuda")
    st, destroy = new_stream()
    torch.cuda.synchronize()
    rra.sparse_encode(x[:5000], 0.5, hdr, vals, idx, stream=st)
    rra.sparse_decode(hdr, vals, idx, 5000, back, stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        for call in (lambda: rra.sparse_encode(x, 0.5, hdr, vals, idx),
                     lambda: rra.sparse_decode(hdr, vals, idx, x.numel(), back)):
            with pytest.raises(rra.RRAError):
                call()
        rra.sparse_encode(x[:5000], 0.5, hdr, vals, idx)
        y.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 1).all() and torch.equal(back[:5000], x[:5000])
    assert hdr.tolist() == [1, int((x[:5000] != 0).sum())]
    destroy()
