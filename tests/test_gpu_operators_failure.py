"""The grouped products' bounded waits, without a GPU fault: with the bound set to 0 the
products give up at their first wait, with copies in flight; the kernel records the timeout, lets its copies and
products end, frees its tensor memory and returns, and the next call is right again."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad", "mx_forward"])
def test_wait_bound_reports_timeout_and_context_survives(op):
    from expert_routed_ffn_gb300 import build
    build.build()
    gen = torch.Generator(device="cuda").manual_seed(61)
    counts, N, K = [70, 0, 333, 19], 512, 1024
    offs = torch.tensor([0, 70, 70, 403, 422], dtype=torch.int32, device="cuda")
    X, dY, W = (torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16) for s in ((422, K), (422, N), (4, N, K)))
    Xq, Wq = capi.mx_quantize(X, "mxfp4"), capi.mx_quantize(W, "mxfp4")
    call = {"forward": lambda: capi.grouped_forward(X, W, offs), "dgrad": lambda: capi.grouped_dgrad(dY, W, offs),
            "wgrad": lambda: capi.grouped_wgrad(dY, X, offs), "mx_forward": lambda: capi.mx_grouped_forward(*Xq, *Wq, offs)}[op]
    want = call()
    assert capi.operators_status() == capi.MOE_OK
    lib = capi.load()
    capi.check(lib.moe_operators_wait_limit(0), "moe_operators_wait_limit")
    try:
        call()
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
        assert "bound" in lib.moe_last_error().decode()
    finally:
        capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
    assert torch.equal(call(), want)
    assert capi.operators_status() == capi.MOE_OK
