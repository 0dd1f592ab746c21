"""Workspaces and captured graphs.

A graph goes on using the workspace memory it was captured with: a Workspace
that grows afterwards keeps it.  And a buffer made inside a capture is zeroed only
by that graph, so other graphs and eager calls get their own.
"""
import gc
import weakref
from unittest import mock

import pytest
import torch


class Host:
    """A Workspace on host memory whose queries give their argument; `capture` is what its stream is in."""

    def __init__(self, larosa):
        self.capture = 0
        self.larosa = larosa
        self.ws = larosa.Workspace("cpu")

    def get(self, nbytes):
        lib = mock.Mock(bytes_of=lambda n: n)
        with mock.patch.object(torch.cuda, "device"), mock.patch.object(self.larosa, "_lib", lib), \
                mock.patch.object(self.larosa, "_capture_id", lambda device: self.capture):
            return self.ws._sized(("bytes_of", nbytes))


def test_a_buffer_that_was_outgrown_stays():
    from activation_sparsity_b200 import larosa
    h = Host(larosa)
    h.get(100)[:] = 1
    first = weakref.ref(h.ws.buf)
    for n in (101, 150, 1000, 1001):
        h.get(n)
    gc.collect()
    assert first() is not None and first().numel() == 100
    kept = [b.numel() for b in h.ws._outgrown]
    assert sum(kept) <= h.ws.buf.numel() and h.ws.buf.numel() <= 2 * 1001 and not h.ws.buf.any()
    h.ws.reset()
    assert not first().any()


def test_a_buffer_made_in_a_capture_serves_that_capture_alone():
    from activation_sparsity_b200 import larosa
    h = Host(larosa)
    h.capture = 7
    a = h.get(100)
    assert h.get(60) is a
    h.capture = 9
    b = h.get(80)
    assert b is not a and h.get(100) is b
    h.capture = 0
    c = h.get(50)
    assert c is not a and c is not b and h.get(100) is c
    h.capture = 11
    assert h.get(100) is c  # made outside of any capture: zero before every one
    d = h.get(500)
    h.capture = 0
    assert h.get(500) is not d


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def decode(L, seed):
    """A one-token call with a 4-bit weight whose splits meet in the workspace, and its inputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(1, 4096, generator=g, device="cuda")
    W = L.larosa_mx4_quantize(torch.randn(4096, 1024, generator=g, device="cuda"), axis=0)
    return x, W


@pytest.mark.gpu
def test_a_graph_keeps_its_memory_when_its_workspace_grows(L):
    x, W = decode(L, 1)
    ws = L.Workspace()
    want = L.larosa_mx4_topk_linear(x, *W, 2000, ws=ws).clone()
    size = ws.buf.numel()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = L.larosa_mx4_topk_linear(x, *W, 2000, ws=ws)
    p = L.larosa_mx4_quantize(torch.randn(3000, 4096, device="cuda"))
    Wt = L.larosa_mx4_quantize(torch.randn(4096, 4096, device="cuda"))
    L.larosa_mx4_linear(*p, *Wt, ws=ws)  # a prompt: a larger workspace
    assert ws.buf.numel() > size
    torch.cuda.synchronize()
    # what would lie where the graph's workspace was, had it been given back
    others = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert all(torch.all(o == 0x5A) for o in others)


@pytest.mark.gpu
def test_graphs_captured_on_one_stream_do_not_depend_on_one_another(L):
    """Workspaces left to the library: two graphs of one capture stream, the second replayed first, then
    an eager call on that stream."""
    x, W = decode(L, 2)
    want = L.larosa_mx4_topk_linear(x, *W, 2000).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = L.larosa_mx4_topk_linear(x, *W, 2000)
            z = L.larosa_mx4_topk_linear(x, *W, 2000)
        graphs.append((g, y, z))
    with torch.cuda.stream(s):
        eager = L.larosa_mx4_topk_linear(x, *W, 2000)
    s.synchronize()
    assert torch.equal(eager, want)
    for g, y, z in reversed(graphs):
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(z, want)
