"""Operators, and the block, one directly behind the other on a stream: each lets the next kernel
start early, which may then read only after its wait what the one before writes.  Every chain is run
without a pause, on buffers that hold something else before, and compared with itself run in steps."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi
from expert_routed_ffn_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.mark.parametrize("norm", ["rms", "gemma"])
@pytest.mark.parametrize("T", [1, 150])
def test_norm_weights_written_by_the_operator_before(T, norm):
    shape = wl.NANO_DECODE.replace(name="norm_chain", T=T, num_experts=16, mlp_norm=norm)
    inputs = wl.make_inputs(shape, "cuda")
    gen = torch.Generator(device="cuda").manual_seed(101)
    values = [torch.randn(shape.H, generator=gen, device="cuda") for _ in range(4)]
    rest = torch.randn(20_000_000, generator=gen, device="cuda")  # keeps the operator's CTAs busy
    into = torch.empty_like(rest)
    blk = capi.block_from_inputs(shape, inputs)
    want = []
    for v in values:
        capi.clip_grad_norm([v, rest], 1e9, out=[inputs["pre_norm_w"], into])
        torch.cuda.synchronize()
        want.append(blk.forward(inputs["X"]))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    got = []
    for _ in range(5):
        for v in values:
            capi.clip_grad_norm([v, rest], 1e9, out=[inputs["pre_norm_w"], into])
            got.append(blk.forward(inputs["X"]))
    torch.cuda.synchronize()
    assert blk.sync_status() == capi.MOE_OK
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4]), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [3, 500, 24576])
def test_tensors_rewritten_between_the_operators(rows, dtype):
    """One buffer that every operator's result goes to and the next one reads, many rounds without a
    pause and as a captured graph."""
    K, N = 512, 512
    gen = torch.Generator(device="cuda").manual_seed(102)
    W = torch.randn(2, N, K, generator=gen, device="cuda").mul_(0.06).to(torch.bfloat16)
    Wq = capi.mx_quantize(W, "mxfp4")
    offs = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    start = torch.randn(rows, K, generator=gen, device="cuda").to(torch.bfloat16)
    codes, scales = capi.mx_quantize(start, "mxfp4")
    X, Y, dW = torch.empty_like(start), torch.empty(rows, N, dtype=dtype, device="cuda"), torch.empty(2, N, K, device="cuda")

    def step(pause):
        for call in (
                lambda: capi.mx_quantize(Y, "mxfp4", codes=codes, scales=scales),
                lambda: capi.mx_dequantize(codes, scales, "mxfp4", out=X),
                lambda: capi.grouped_forward(X, W, offs, out=Y),
                lambda: capi.clip_grad_norm([Y], 3.0 * rows ** 0.5),
                lambda: capi.mx_quantize(Y, "mxfp4", codes=codes, scales=scales),
                lambda: capi.mx_grouped_forward(codes, scales, *Wq, offs, out=Y),
                lambda: capi.mx_quantize(Y, "mxfp8", codes=codes8, scales=scales),
                lambda: capi.mx_dequantize(codes8, scales, "mxfp8", out=X),
                lambda: capi.grouped_wgrad(X, X, offs, out=dW),
                lambda: capi.grouped_dgrad(X, W, offs, out=Y)):
            call()
            if pause:
                torch.cuda.synchronize()

    codes8 = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    want = []
    Y.copy_(start)
    for _ in range(6):
        step(True)
        want.append((Y.clone(), dW.clone()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(False)
    for run in (lambda: step(False), graph.replay):
        for _ in range(3):
            X.fill_(float("nan"))
            dW.fill_(float("nan"))
            Y.copy_(start)
            got = []
            for _ in range(6):
                run()
                got.append((Y.clone(), dW.clone()))
            torch.cuda.synchronize()
            for i, (g, w) in enumerate(zip(got, want)):
                assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]), i
    assert capi.operators_status() == capi.MOE_OK
    assert bool(want[-1][0].isfinite().all()) and float(want[-1][0].float().abs().max()) > 0
