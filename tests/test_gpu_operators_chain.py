"""The operators used together, as a program around the block would: routing and dispatch by
the block, the experts' MLP product by product, its gradients, clipping, and the MXFP4 form.

The chain's own rounding points (bf16 hidden activations and gradients between products) are
put into the fp64 reference where they occur, so each product is held to its own bound."""

import ctypes

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


def _dispatch(idx, E):
    T, k = idx.shape
    offs = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    token, slot = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    bad = torch.empty(1, dtype=torch.int32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = capi.load().moe_dispatch_noalloc(p(idx), T, k, E, p(offs), p(token), p(slot), p(bad),
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == capi.MOE_OK
    return offs, token.long(), slot.long()


SHAPE = wl.NANO_DECODE.replace(name="chain", T=150, num_experts=32, num_shared_experts=0, shared_intermediate_size=0)


def _silu_mul(g, u):
    return torch.nn.functional.silu(g) * u


def test_products_make_the_block():
    inputs = wl.make_inputs(SHAPE, "cuda")
    blk = capi.block_from_inputs(SHAPE, inputs)
    X = inputs["X"]
    Y = blk.forward(X).float()
    idx, w = blk.route(X)
    offs, token, slot = _dispatch(idx, SHAPE.E)
    xs = X[token]
    g = capi.grouped_forward(xs, inputs["gate"], offs, out_dtype=torch.float32)
    u = capi.grouped_forward(xs, inputs["up"], offs, out_dtype=torch.float32)
    h = _silu_mul(g, u).to(torch.bfloat16)
    y = capi.grouped_forward(h, inputs["down"], offs, out_dtype=torch.float32)
    mine = (y[slot].view(SHAPE.T, SHAPE.k, -1) * w.unsqueeze(-1)).sum(1)
    # the block's hidden activations are rounded to bf16 from a fast exponential, so one may fall
    # on the other bf16 neighbour: both are within the block's bound of the exact result
    assert float((mine - Y).abs().max()) <= 2 * 2e-2 * float(Y.square().mean().sqrt())
    assert capi.operators_status() == capi.MOE_OK and blk.sync_status() == capi.MOE_OK


def test_training_step_of_the_experts():
    """Gradients of sum(G * mlp(x)) by x and the three weights against autograd in fp64, then clipped."""
    inputs = wl.make_inputs(SHAPE, "cuda")
    blk = capi.block_from_inputs(SHAPE, inputs)
    idx, _ = blk.route(inputs["X"])
    offs, token, _ = _dispatch(idx, SHAPE.E)
    xs = inputs["X"][token]
    gate, up, down = inputs["gate"], inputs["up"], inputs["down"]
    G = torch.randn(xs.shape, generator=torch.Generator(device="cuda").manual_seed(51), device="cuda").to(torch.bfloat16)

    g = capi.grouped_forward(xs, gate, offs, out_dtype=torch.float32)
    u = capi.grouped_forward(xs, up, offs, out_dtype=torch.float32)
    h = _silu_mul(g, u).to(torch.bfloat16)
    dh = capi.grouped_dgrad(G, down, offs, out_dtype=torch.float32)
    d_down = capi.grouped_wgrad(G, h, offs)
    s = torch.sigmoid(g)
    dg = (dh * u * s * (1 + g * (1 - s))).to(torch.bfloat16)
    du = (dh * g * s).to(torch.bfloat16)
    dx = capi.grouped_dgrad(dg, gate, offs, out_dtype=torch.float32) + capi.grouped_dgrad(du, up, offs, out_dtype=torch.float32)
    d_gate, d_up = capi.grouped_wgrad(dg, xs, offs), capi.grouped_wgrad(du, xs, offs)

    x64 = xs.double().requires_grad_()
    leaves = [t.double().requires_grad_() for t in (gate, up, down)]
    o = offs.tolist()
    out = torch.cat([_silu_mul(x64[a:b] @ leaves[0][e].t(), x64[a:b] @ leaves[1][e].t()) @ leaves[2][e].t()
                     for e, (a, b) in enumerate(zip(o[:-1], o[1:]))])
    want = torch.autograd.grad((out * G.double()).sum(), [x64, *leaves])
    for got, ref in zip((dx, d_gate, d_up, d_down), want):
        # one bf16 rounding (2^-8 of a value at most) of h, dg or du enters each sum: 2^-8 of its norm
        assert float((got.double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
    grads = [d_gate, d_up, d_down]
    norm = float(torch.stack([t.norm() for t in want[1:]]).norm())
    before = [t.clone() for t in grads]
    got = float(capi.clip_grad_norm(grads, norm / 4))
    assert abs(got - norm) <= 2.0 ** -8 * norm
    for t, b in zip(grads, before):
        assert float((t - b * (norm / 4 / got)).abs().max()) <= 2.0 ** -18 * float(b.abs().max())
    assert capi.operators_status() == capi.MOE_OK


def test_mxfp4_experts():
    """Quantised tokens and weights through dispatch offsets: equal to the bf16 product of the decoded values."""
    inputs = wl.make_inputs(SHAPE, "cuda")
    blk = capi.block_from_inputs(SHAPE, inputs)
    idx, _ = blk.route(inputs["X"])
    offs, token, _ = _dispatch(idx, SHAPE.E)
    W = capi.mx_quantize(inputs["gate"], "mxfp4")
    X = capi.mx_quantize(inputs["X"][token], "mxfp4")
    got = capi.mx_grouped_forward(*X, *W, offs, out_dtype=torch.float32)
    x, w = capi.mx_dequantize(*X, "mxfp4"), capi.mx_dequantize(*W, "mxfp4")  # exact in bf16
    want = capi.grouped_forward(x, w, offs, out_dtype=torch.float32)
    mag = capi.grouped_forward(x.abs(), w.abs(), offs, out_dtype=torch.float32)
    assert bool(((got - want).abs() <= 2 * SHAPE.H * 2.0 ** -23 * mag).all())
    assert capi.operators_status() == capi.MOE_OK
