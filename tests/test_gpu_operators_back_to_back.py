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
