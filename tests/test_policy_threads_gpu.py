"""Calls of the losses over a vocabulary from several host threads, and of several sizes in one
captured graph."""
import ctypes
import threading

import pytest
import torch

import segmented_associative_scan_gb300 as rlca
from segmented_associative_scan_gb300 import policy as pol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    rlca.build()


# Rows that are parked in 43, 67 and 104 KB of shared memory.
SIZES = (22000, 34000, 53000)


def inputs(V, seed, rows=70):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, 1, V, generator=g).to(torch.bfloat16).cuda()
    tokens = torch.randint(0, V, (rows, 1), generator=g).cuda()
    old, adv = (torch.randn(rows, 1, generator=g).cuda() for _ in range(2))
    return z, tokens, old, adv


def structures(args, out):
    """The C structures of a call, for calls without the binding's work between them."""
    z, tokens, old, adv = args
    (N, T, V), line = z.shape, lambda t: pol.Line(t.data_ptr(), 1)
    steps = lambda t: pol.Steps(t.data_ptr(), V, V)
    p = pol.Choices(N, T, V, steps(z), tokens.data_ptr(), 1, None, 8, 1.0)
    q = pol.Policy(line(old), line(adv), pol.Line(None, 0), pol.Line(None, 0), 0.2, 0.2, 0.0, 0.0,
                   out[0].data_ptr(), out[1].data_ptr(), None, None, steps(out[4]))
    return p, q


def test_threads_with_different_vocabularies(cuda_device):
    """Threads that call at the same time, each on a stream of its own and with a vocabulary of its own:
    no call fails, and each gives what it gives alone."""
    work = [inputs(V, i) for i, V in enumerate(SIZES + SIZES[::2])]
    want = [rlca.policy_loss(*w, want_grad=True) for w in work]
    outs = [[None if t is None else torch.zeros_like(t) for t in w] for w in want]
    calls = [structures(w, o) for w, o in zip(work, outs)]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    fn = rlca.lib().rlca_policy_loss_bf16
    statuses = [set() for _ in work]
    start = threading.Barrier(len(work))

    def thread(i):
        p, q = (ctypes.byref(x) for x in calls[i])
        stream = streams[i].cuda_stream
        start.wait()
        for _ in range(20000):
            statuses[i].add(fn(p, q, stream))

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{0}] * len(work)
    for got, expect in zip(outs, want):
        assert torch.equal(got[0], expect[0]) and torch.equal(got[4], expect[4])


def test_different_vocabularies_in_one_graph(cuda_device):
    work = [inputs(V, 7 + i) for i, V in enumerate(SIZES)]
    work += work[::-1]
    want = [rlca.policy_loss(*w, want_grad=True) for w in work]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [rlca.policy_loss(*w, want_grad=True) for w in work]
    for _ in range(2):
        for t in got:
            t[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[4], b[4])
