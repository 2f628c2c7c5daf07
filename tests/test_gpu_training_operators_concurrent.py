"""Calls of the training operators that overlap: on two streams, from two threads, and as two captured
graphs replayed side by side; each gives what it gives alone."""

import threading

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


class Work:
    """One of each, on tensors of its own."""

    def __init__(self, seed, rows, I, K, T, H, sides):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def bf(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(BF)

        self.X, self.dY = bf(rows, K), bf(rows, K)
        self.Wg, self.Wu, self.Wd = bf(3, I, K, std=0.1), bf(3, I, K, std=0.1), bf(3, K, I, std=0.1)
        self.offs = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
        self.S, self.F = torch.randn(T, H, generator=gen, device="cuda"), bf(T, H)
        self.how = dict(pre_w=torch.rand(H, generator=gen, device="cuda"), post_w=torch.rand(H, generator=gen, device="cuda"),
                        gate=torch.rand(T, 1, generator=gen, device="cuda"))
        self.G = torch.randn(*sides, generator=gen, device="cuda")

    def run(self):
        H, G, U = capi.grouped_gated_forward(self.X, self.Wg, self.Wu, self.offs, save=True)
        dG, dU = capi.grouped_gated_backward(self.dY, self.Wd, G, U, self.offs)
        dX = capi.grouped_gated_dgrad(dG, dU, self.Wg, self.Wu, self.offs)
        new, N = capi.sandwich_norm(self.S, self.F, **self.how)
        back = capi.sandwich_norm_backward(self.S, N, new, self.F, **self.how)
        return [H, G, U, dG, dU, dX, new, N, *back, capi.orthogonalize(self.G)]


def _two():
    return Work(61, 500, 200, 328, 700, 1024, (3, 264, 136)), Work(62, 77, 1408, 256, 33, 6144, (1, 520, 1032))


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams():
    works = _two()
    want = [w.run() for w in works]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    got = [[], []]
    for _ in range(10):
        for w, s, g in zip(works, streams, got):
            with torch.cuda.stream(s):
                g.append(w.run())
    torch.cuda.synchronize()
    assert all(_same(r, want[i]) for i in range(2) for r in got[i])


def test_two_threads():
    works = _two()
    want = [w.run() for w in works]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def loop(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i].append(works[i].run())
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and all(len(g) == 10 for g in got)
    assert all(_same(r, want[i]) for i in range(2) for r in got[i])


def test_two_graphs_side_by_side():
    works = _two()
    want = [w.run() for w in works]
    torch.cuda.synchronize()
    graphs, got = [], []
    for w in works:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(w.run())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in works]
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(_same(got[i], want[i]) for i in range(2))
