"""The norms' bounded wait for a row, without a GPU fault: with the bound set to 0 every team gives up at its
first row, with copies in flight; the kernel records the timeout, waits for its copies and returns, what it
read is as it was, and the next call is right again."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


def _gives_up(call):
    lib = capi.load()
    capi.check(lib.moe_operators_wait_limit(0), "moe_operators_wait_limit")
    try:
        call()
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
        assert "bound" in lib.moe_last_error().decode()
    finally:
        capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")


@pytest.mark.parametrize("without", [(), ("post_w",), ("pre_w",), ("pre_w", "post_w"), ("F", "post_w", "gate")])
@pytest.mark.parametrize("T,H,x_type,f_type,gate", [(1, 8, BF, BF, "token"), (3, 2048, F32, BF, "channel"), (5000, 264, BF, BF, "token"),
                                                    (2000, 1408, F32, BF, "channel"), (700, 8192, F32, F32, "channel")])
def test_wait_bound_of_zero_gives_up(T, H, x_type, f_type, gate, without):
    gen = torch.Generator(device="cuda").manual_seed(81)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"X": randn(T, H).to(x_type), "F": randn(T, H).to(f_type), "pre_w": randn(H), "post_w": randn(H),
         "gate": randn(T, 1) if gate == "token" else randn(H), "dX": randn(T, H).to(x_type), "dN": randn(T, H).to(f_type)}
    for name in without:
        s[name] = None
    if s["pre_w"] is None:
        s["dN"] = None
    kept = {k: v.clone() for k, v in s.items() if v is not None}
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"], residual_scale=0.5)

    def forward():
        return [t for t in capi.sandwich_norm(s["X"], s["F"], **how) if t is not None]

    def backward():
        return [t for t in capi.sandwich_norm_backward(s["dX"], s["dN"], s["X"], s["F"], **how) if t is not None]

    for call in (forward, backward):
        want = call()
        assert capi.operators_status() == capi.MOE_OK
        _gives_up(call)
        assert all(torch.equal(s[k], v) for k, v in kept.items())
        again = call()
        assert capi.operators_status() == capi.MOE_OK
        assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_a_captured_call_keeps_its_bound():
    X = torch.ones(400, 1024, dtype=BF, device="cuda")
    w = torch.ones(1024, device="cuda")
    want = capi.sandwich_norm(X, X.clone(), pre_w=w, post_w=w)
    F = X.clone()
    lib, graphs = capi.load(), []
    for bound in (0, -1):
        capi.check(lib.moe_operators_wait_limit(bound), "moe_operators_wait_limit")
        graph = torch.cuda.CUDAGraph()
        try:
            with torch.cuda.graph(graph):
                out = capi.sandwich_norm(X, F, pre_w=w, post_w=w)
        finally:
            capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
        graphs.append((graph, out))
    graphs[0][0].replay()
    assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
    graphs[1][0].replay()
    assert capi.operators_status() == capi.MOE_OK
    assert all(torch.equal(a, b) for a, b in zip(graphs[1][1], want))
