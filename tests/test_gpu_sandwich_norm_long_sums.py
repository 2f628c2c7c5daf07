"""The norms' sums over many rows: the gradients of weights and of a channel's gate.

A team adds up to 1024 rows one after the other, a CTA up to 16 teams; the CTAs' sums are added in 32
compensated sums (2 u and second-order terms) and those one after the other: off by at most 1075 u of the sum
of magnitudes (u = 2^-24), whatever the number of rows.  The terms' own errors as tests/test_gpu_sandwich_norm.py derives them (r = 32 u).
"""

import ctypes

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
R = 32 * U
SUM = 1075 * U
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()
    assert capi.operators_status() == capi.MOE_OK


def _close(got, ref, err):
    bound = 1.01 * err + torch.finfo(got.dtype).eps / 2 * (ref.abs() + err)
    assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() / bound).max())


@pytest.mark.parametrize("T", [1_000_000, 40_000_000])
def test_rows_alike(T):
    """The same term from each row, 4.4e-4 from what fp32 holds beside a sum of 8192 of them or more: one chain of
    40000000 / (152 * 16) such additions is 2e-4 off, more than the bound."""
    H, eps = 8, 0.9 * 2.0 ** -10
    one = torch.ones(T, H, dtype=BF, device="cuda")
    w, gate = torch.ones(H, device="cuda"), torch.ones(H, device="cuda")
    dX, dF, dpre, dpost, dgate = capi.sandwich_norm_backward(one, one, one, one, pre_w=w, post_w=w, gate=gate, eps=eps)
    hat = 1 / (1 + ctypes.c_float(eps).value) ** 0.5  # of every value of both norms
    t = 1 + hat * (1 - hat * hat)
    # T's error: rx (|xh| d(m) + (|dN w| + |xh m|) (r + 8 u)) + 4 u (|dX'| + rx (|dN w| + |xh m|)), all factors about one
    dt = 1.01 * ((48 * U + R + 6 * U) + 2 * (R + 8 * U) + 4 * U * 3)
    ref = torch.full((H,), T, dtype=torch.float64, device="cuda")
    _close(dpre, ref * hat, T * hat * (R + 2 * U + SUM))
    for got in (dpost, dgate):
        _close(got, ref * t * hat, T * (dt + 1.01 * (R + 4 * U) + 1.01 * SUM))


@pytest.mark.parametrize("T,H,gate", [(400_000, 6144, "channel"), (400_000, 1032, "none"), (3_000_001, 136, "token"), (157_000, 8192, "channel")])
def test_random_rows(T, H, gate):
    gen = torch.Generator(device="cuda").manual_seed(91)

    def rows(scale):
        t = torch.empty(T, H, dtype=BF, device="cuda")
        for i in range(0, T, 50_000):
            t[i:i + 50_000] = torch.randn(t[i:i + 50_000].shape, generator=gen, device="cuda") * scale
        return t

    X, F, dX, dN = rows(1.0), rows(3.0), rows(0.5), rows(1.0)
    w, v = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda") for _ in range(2))
    g = {"none": None, "token": torch.randn(T, 1, generator=gen, device="cuda"), "channel": torch.randn(H, generator=gen, device="cuda")}[gate]
    got = capi.sandwich_norm_backward(dX, dN, X, F, pre_w=w, post_w=v, gate=g)
    again = capi.sandwich_norm_backward(dX, dN, X, F, pre_w=w, post_w=v, gate=g)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
    sums = {k: torch.zeros(H, dtype=torch.float64, device="cuda") for k in ("pre", "dpre", "post", "dpost", "gate", "dgate")}
    for i in range(0, T, 20_000):
        part = slice(i, i + 20_000)
        x, f, dx, dn = (t[part].double() for t in (X, F, dX, dN))
        rx, rf = (1 / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-5) for t in (x, f))
        xh, fh, back = x * rx, f * rf, dn * w.double()
        m = (back * xh).mean(-1, keepdim=True)
        terms = back.abs() + (xh * m).abs()
        dt = rx * (xh.abs() * (48 * U * (back * xh).abs().mean(-1, keepdim=True) + m.abs() * (R + 6 * U)) + terms * (R + 8 * U)) \
            + 4 * U * (dx.abs() + rx * terms)
        t = dx + rx * (back - xh * m)
        by = torch.ones(1, dtype=torch.float64, device="cuda") if g is None else g[part].double() if gate == "token" else g.double()
        sums["pre"] += (dn * xh).sum(0)
        sums["dpre"] += (dn * xh).abs().sum(0) * (R + 2 * U + SUM)
        sums["post"] += (t * by * fh).sum(0)
        sums["dpost"] += (dt * (by * fh).abs() + (t * by * fh).abs() * (R + 4 * U + SUM)).sum(0)
        sums["gate"] += (t * fh * v.double()).sum(0)
        sums["dgate"] += (dt * (fh * v.double()).abs() + (t * fh * v.double()).abs() * (R + 4 * U + SUM)).sum(0)
    _close(got[2], sums["pre"], sums["dpre"])
    _close(got[3], sums["post"], sums["dpost"])
    if gate == "channel":
        _close(got[4], sums["gate"], sums["dgate"])


@pytest.mark.parametrize("H", [8, 264, 2048, 4104, 8192])
def test_workspace_holds_the_partial_sums(H):
    """The call writes its partial sums inside the workspace it asked for, around the numbers of rows where the
    number of CTAs grows."""
    lib = capi.load()
    teams = {8: 16, 264: 16, 2048: 4, 4104: 1, 8192: 1}[H]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for T in (1, 255, 256, 257, 1024 * teams * sms, 1024 * teams * sms + 1):
        if T * H > 1 << 31:
            continue
        need = ctypes.c_size_t()
        assert lib.moe_sandwich_norm_workspace(T, H, ctypes.byref(need)) == capi.MOE_OK
        pool = torch.full((need.value + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        X = torch.ones(T, H, dtype=BF, device="cuda")
        out, w, dw = torch.empty_like(X), torch.ones(H, device="cuda"), torch.empty(H, device="cuda")
        status = lib.moe_sandwich_norm_backward(None, X.data_ptr(), X.data_ptr(), None, w.data_ptr(), None, None, 0, 1.0, 1e-5, 1, T, H, 0, 0,
                                                out.data_ptr(), None, dw.data_ptr(), None, None, pool.data_ptr(), need.value,
                                                torch.cuda.current_stream().cuda_stream)
        assert status == capi.MOE_OK and bool((pool[need.value:] == 0x5A).all())
        hat = 1 / (1 + ctypes.c_float(1e-5).value) ** 0.5
        _close(dw, torch.full_like(dw, T * hat, dtype=torch.float64), T * hat * (R + 2 * U + SUM))
