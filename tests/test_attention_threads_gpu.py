"""Calls, errors and status calls of several host threads on one stream."""

import ctypes
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402


class Split:
    """Attention whose units are split over blocks and joined by a second kernel, called through the C ABI
    (which lets threads run side by side)."""

    def __init__(self, q_heads, threads, calls, n=20000):
        g = torch.Generator(device="cuda")
        g.manual_seed(6)
        page, heads, dim = 64, 2, 64
        pages = -(-(n + 1) // page)
        self.k, self.v = (torch.randn(pages, page, heads, dim, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
        self.table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        self.ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.q = torch.randn(threads, calls, 1, 1, q_heads, dim, device="cuda", generator=g).to(torch.bfloat16)
        self.want = torch.stack([torch.stack([tks.tree_attention(q, self.k, self.v, self.table, self.ctx) for q in row]) for row in self.q])
        self.out = torch.zeros_like(self.q)
        self.cache = tks.Cache(self.k.data_ptr(), self.v.data_ptr(), None, tks.TKS_BF16, pages, page, heads, dim, *self.k.stride()[:3])
        self.slots = pages * page
        torch.cuda.synchronize()

    def call(self, i, j, stream):
        heads, dim = self.q.shape[4:]
        q = tks.Queries(self.q[i, j].data_ptr(), heads * dim, heads * dim, dim, self.out[i, j].data_ptr(), None, 1, 1, heads,
                        self.table.data_ptr(), self.table.shape[1], self.table.shape[1], dim ** -0.5)
        return tks.load().tks_tree_attention(ctypes.byref(self.cache), ctypes.byref(q), self.ctx.data_ptr(), None, None, stream)


def together(*runs):
    """Runs them in a thread each; an exception of any is raised here."""
    failed = []

    def guarded(run):
        try:
            run()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=guarded, args=(r,)) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("q_heads", [4, 80])
def test_status_calls_between_other_threads_calls(q_heads):
    """One thread makes an error and asks for it, over and over: it is told each one, and the others' results are whole."""
    threads, calls = 3, 100
    case = Split(q_heads, threads, calls)
    stream = torch.cuda.Stream().cuda_stream
    bad = torch.tensor([case.slots], dtype=torch.int32, device="cuda")
    rows = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    rcs, told = [], []

    def errors():
        for _ in range(calls):
            rcs.append(tks.load().tks_cache_read(ctypes.byref(case.cache), bad.data_ptr(), 1, rows[0].data_ptr(), rows[1].data_ptr(), tks.TKS_BF16, stream))
            told.append(tks.load().tks_device_status(stream))

    together(errors, *(lambda i=i: [rcs.append(case.call(i, j, stream)) for j in range(calls)] for i in range(threads)))
    torch.cuda.synchronize()
    assert rcs == [tks.TKS_OK] * (calls * (threads + 1))
    assert told == [tks.TKS_E_INDEX] * calls
    assert tks.load().tks_device_status(stream) == tks.TKS_OK
    assert torch.equal(case.out, case.want)


def test_no_report_is_lost_between_status_calls():
    """One thread makes errors while another asks: each error is told by a status call that ended after it was made."""
    case = Split(4, 1, 60)
    stream = torch.cuda.Stream().cuda_stream
    bad = torch.tensor([case.slots], dtype=torch.int32, device="cuda")
    rows = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    told, made, done = [], [], threading.Event()

    def errors():
        for _ in range(40):
            made.append(len(told))
            assert tks.load().tks_cache_read(ctypes.byref(case.cache), bad.data_ptr(), 1, rows[0].data_ptr(), rows[1].data_ptr(), tks.TKS_BF16, stream) == tks.TKS_OK
        done.set()

    def ask():
        while not done.is_set():
            told.append(tks.load().tks_device_status(stream))
        told.append(tks.load().tks_device_status(stream))

    together(errors, ask, lambda: [case.call(0, j, stream) for j in range(60)])
    assert len(made) == 40 and set(told) <= {tks.TKS_OK, tks.TKS_E_INDEX}
    assert all(tks.TKS_E_INDEX in told[at:] for at in made)
    assert tks.load().tks_device_status(stream) == tks.TKS_OK
    torch.cuda.synchronize()
    assert torch.equal(case.out, case.want)


@pytest.mark.parametrize("q_heads", [4, 80])
def test_the_per_thread_stream(q_heads):
    """One handle, a stream of its own in every thread: the calls run side by side, and each thread has its own errors."""
    threads, calls, per_thread = 4, 50, 2  # (the handle's value: cudaStreamPerThread)
    case = Split(q_heads, threads, calls)
    bad = torch.tensor([case.slots], dtype=torch.int32, device="cuda")
    rows = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    rcs, told = [], {}
    begin = threading.Barrier(threads)

    def run(i):
        begin.wait()
        rcs.extend(case.call(i, j, per_thread) for j in range(calls))
        if i == 0:
            rcs.append(tks.load().tks_cache_read(ctypes.byref(case.cache), bad.data_ptr(), 1, rows[0].data_ptr(), rows[1].data_ptr(), tks.TKS_BF16, per_thread))
        begin.wait()
        told[i] = tks.load().tks_device_status(per_thread)

    together(*(lambda i=i: run(i) for i in range(threads)))
    assert rcs == [tks.TKS_OK] * (threads * calls + 1)
    assert told == {0: tks.TKS_E_INDEX, 1: tks.TKS_OK, 2: tks.TKS_OK, 3: tks.TKS_OK}
    torch.cuda.synchronize()
    assert torch.equal(case.out, case.want)
