"""The grouped products' bounded waits under work that is long but sound: with a bound far above
every single wait and far below the kernel's run time, no wait may run out."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,N,K", [
    ([64] * 254 + [33], 2048, 2048),            # one stage a tile, then a tail
    ([64] * 100 + [0] * 100 + [33, 48, 17], 2048, 2048),
    ([2048] * 60 + [1, 2048, 2047], 1024, 1024),  # many stages a tile
])
def test_wgrad_with_a_tail_behind_many_tiles_without(counts, N, K):
    """Only the last experts' row counts leave a tail to zero: the warp that does so has nothing to
    wait for until then."""
    from expert_routed_ffn_gb300 import build
    build.build()
    lib = capi.load()
    gen = torch.Generator(device="cuda").manual_seed(91)
    rows = sum(counts)
    dY, X = (torch.randn(rows, n, generator=gen, device="cuda").to(torch.bfloat16) for n in (N, K))
    offs = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device="cuda")
    out = torch.empty(len(counts), N, K, device="cuda")
    capi.grouped_wgrad(dY, X, offs, out=out)  # the first call also loads the kernel
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    capi.grouped_wgrad(dY, X, offs, out=out)
    end.record()
    assert capi.operators_status() == capi.MOE_OK
    want, us = out.clone(), start.elapsed_time(end) * 1e3
    assert us > 133  # the bound below, at 1.5 GHz (97 us at 2.07)
    capi.check(lib.moe_operators_wait_limit(200_000), "moe_operators_wait_limit")
    try:
        out.fill_(-1)
        capi.grouped_wgrad(dY, X, offs, out=out)
        assert capi.operators_status() == capi.MOE_OK
    finally:
        capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad", "accumulate", "mx_forward"])
def test_timeout_in_a_sum_of_several_segments(op, dtype):
    """The bound at 0: the products give up at their first wait, report it, and the next call is right."""
    from expert_routed_ffn_gb300 import build
    build.build()
    lib = capi.load()
    gen = torch.Generator(device="cuda").manual_seed(92)
    long, counts = 70_016, [33, 0, 90, 5]
    if op in ("wgrad", "accumulate"):
        counts = [33, 70_017, 0, 5]
    rows, N, K = sum(counts), 136, 264
    if op in ("forward", "mx_forward"):
        K = long
    elif op == "dgrad":
        N = long
    offs = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(4)], dtype=torch.int32, device="cuda")
    X, dY, W = (torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16) for s in ((rows, K), (rows, N), (4, N, K)))
    if op == "mx_forward":
        Xq, Wq = capi.mx_quantize(X, "mxfp4"), capi.mx_quantize(W, "mxfp4")

    def call():
        if op == "accumulate":
            return capi.grouped_wgrad(dY, X, offs, out=torch.ones(4, N, K, dtype=dtype, device="cuda"), accumulate=True)
        if op == "mx_forward":
            return capi.mx_grouped_forward(*Xq, *Wq, offs, out_dtype=dtype)
        f, a, b = {"forward": (capi.grouped_forward, X, W), "dgrad": (capi.grouped_dgrad, dY, W), "wgrad": (capi.grouped_wgrad, dY, X)}[op]
        return f(a, b, offs, out_dtype=dtype)

    want = call()
    assert capi.operators_status() == capi.MOE_OK
    capi.check(lib.moe_operators_wait_limit(0), "moe_operators_wait_limit")
    try:
        call()
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
    finally:
        capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
    assert torch.equal(call(), want)
    assert capi.operators_status() == capi.MOE_OK


def test_largest_bound():
    """What the roles add to the bound does not overflow it."""
    from expert_routed_ffn_gb300 import build
    build.build()
    lib = capi.load()
    gen = torch.Generator(device="cuda").manual_seed(93)
    counts = [0, 64, 33, 0, 0, 300] * 12
    dY, X = (torch.randn(sum(counts), n, generator=gen, device="cuda").to(torch.bfloat16) for n in (1024, 2048))
    offs = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device="cuda")
    want = capi.grouped_wgrad(dY, X, offs)
    assert capi.operators_status() == capi.MOE_OK
    for limit in (2 ** 63 - 1, 2 ** 62):
        capi.check(lib.moe_operators_wait_limit(limit), "moe_operators_wait_limit")
        try:
            got = capi.grouped_wgrad(dY, X, offs)
            assert capi.operators_status() == capi.MOE_OK
        finally:
            capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
        assert torch.equal(got, want)
