"""moe_mx_quantize / moe_mx_dequantize: exact, so results are compared for equality.

The definition in fp64: the scale is the power of two under the block's largest magnitude
over 2^emax; an element is the nearest value of the element type, a tie going to the one
with the even code; larger ones saturate."""

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


def _element_values(fmt):
    """The element type's non-negative finite values in code order."""
    if fmt == "mxfp4":
        return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)
    return v


def _define(X, fmt):
    """codes (one per element, sign in the top bit of the code) and scale bytes [.., K / 32, rows]."""
    x = X.double().cpu().unflatten(-1, (-1, 32))
    table = _element_values(fmt)
    emax, bits = (2, 3) if fmt == "mxfp4" else (8, 7)
    amax = x.abs().amax(-1)
    finite = torch.isfinite(x).all(-1)
    e = torch.where((amax > 0) & finite, torch.frexp(amax.where(finite, torch.ones(()).double())).exponent - 1 - emax, -127)
    e = e.clamp(min=-127)
    v = (x * torch.exp2(-e.double()).unsqueeze(-1)).where(finite.unsqueeze(-1), torch.zeros((), dtype=torch.float64))
    mid = (table[1:] + table[:-1]) / 2  # exact: neighbours differ in at most a few bits
    a = v.abs()
    low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    code = torch.where(low % 2 == 0, low, high)
    neg = torch.signbit(v) & finite.unsqueeze(-1)
    code = code + (neg.long() << bits)
    scale = torch.where(finite, e + 127, 255)
    return code.flatten(-2).to(torch.uint8), scale.transpose(-1, -2).to(torch.uint8)


def _unpacked(codes, fmt):
    c = codes.cpu()
    return c if fmt == "mxfp8" else torch.stack([c & 15, c >> 4], -1).flatten(-2)


def _values(code, scale, fmt):
    table = _element_values(fmt)
    bits = 3 if fmt == "mxfp4" else 7
    v = table[(code & ((1 << bits) - 1)).long()] * (1 - 2 * (code >> bits).double())
    s = scale.transpose(-1, -2).double()
    e = torch.where(s == 255, torch.full_like(s, float("nan")), torch.exp2(s - 127))
    return (v.unflatten(-1, (-1, 32)) * e.unsqueeze(-1)).flatten(-2)


def _check(X, fmt):
    codes, scales = capi.mx_quantize(X, fmt)
    code, scale = _define(X, fmt)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(_unpacked(codes, fmt), code)
    want = _values(code, scale, fmt)
    for dtype in (torch.float32, torch.bfloat16):
        got = capi.mx_dequantize(codes, scales, fmt, dtype).cpu()
        exact = want.to(torch.float32).to(dtype)  # fp32 holds every value: one rounding
        assert torch.equal(got.isnan(), exact.isnan())
        assert torch.equal(got.nan_to_num(nan=0.0, posinf=1e38, neginf=-1e38), exact.nan_to_num(nan=0.0, posinf=1e38, neginf=-1e38))


SHAPES = [(1, 32), (1, 2048), (3, 96), (63, 288), (64, 256), (65, 32), (130, 1024), (5, 41, 320), (2, 1, 64), (3, 128, 544)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_equals_the_definition(shape, dtype, fmt):
    gen = torch.Generator().manual_seed(21)
    X = torch.randn(shape, generator=gen) * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=gen))
    _check(X.to(dtype).cuda(), fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_ends_and_zeros(dtype, fmt):
    """Every element value and midpoint between two at several scales, both signs, the ends of
    the type, subnormal blocks, zeros of both signs."""
    table = _element_values(fmt)
    points = torch.cat([table, (table[1:] + table[:-1]) / 2, table[-1:] * 1.2]).unique()
    top = table[-1]
    rows = []
    for e in (-126, -100, -3, 0, 5, 100):
        for at in range(0, len(points), 30):
            p = points[at:at + 30]
            row = torch.zeros(32, dtype=torch.float64)
            row[:len(p)] = p * torch.where(torch.arange(len(p)) % 2 == 0, 1.0, -1.0)
            row[30] = top  # fixes the block's scale
            rows.append(row * 2.0 ** e)
    rows += [torch.zeros(32, dtype=torch.float64), -torch.zeros(32, dtype=torch.float64)]
    rows.append(torch.full((32,), float(torch.finfo(torch.bfloat16).max), dtype=torch.float64))
    rows.append(torch.linspace(-1, 1, 32, dtype=torch.float64) * 2.0 ** -127)
    rows.append(torch.linspace(-1, 1, 32, dtype=torch.float64) * 2.0 ** -130)
    _check(torch.stack(rows).to(dtype).cuda(), fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_non_finite_blocks(dtype, fmt):
    X = torch.randn(70, 96, generator=torch.Generator().manual_seed(3))
    X[0, 0], X[1, 33], X[2, 95], X[69, 64] = float("nan"), float("inf"), float("-inf"), -float("nan")
    X = X.to(dtype).cuda()
    _check(X, fmt)
    codes, scales = capi.mx_quantize(X, fmt)
    back = capi.mx_dequantize(codes, scales, fmt)
    assert bool(back[0, :32].isnan().all()) and bool(back[1, 32:64].isnan().all())
    assert int(back.isnan().sum()) == 4 * 32


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_matches_the_checkpoint_layout(fmt):
    """The same codes as the workload generator's, which the block's kernels are tested with."""
    W = torch.randn(192, 512, generator=torch.Generator().manual_seed(4)) * 0.02  # fp32: no exact ties
    want = wl.mx_quantize(W, fmt)
    got = capi.mx_quantize(W.cuda(), fmt)
    assert torch.equal(got[1].cpu(), want[1])
    value = _values(_unpacked(got[0], fmt), want[1], fmt)
    assert torch.equal(value, _values(_unpacked(want[0], fmt), want[1], fmt))


def test_block_runs_on_quantized_weights():
    """moe_create's MXFP4 weights made on the device: the block's outputs are those of the generator's codes."""
    shape = wl.NANO_DECODE.replace(name="nano_q", T=32, weight_format="mxfp4")
    inputs = wl.make_inputs(shape, "cuda")
    plain = wl.make_inputs(shape.replace(weight_format="bf16"), "cuda")
    again = dict(inputs)
    for key in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down"):
        values = capi.mx_dequantize(inputs[key], inputs[f"{key}_scale"], "mxfp4", torch.float32)
        again[key], again[f"{key}_scale"] = capi.mx_quantize(values, "mxfp4")
        assert values.shape == plain[key].shape
    a, b = capi.block_from_inputs(shape, inputs), capi.block_from_inputs(shape, again)
    assert torch.equal(a.forward(inputs["X"]), b.forward(inputs["X"]))


def test_empty_graph_and_stream():
    codes, scales = capi.mx_quantize(torch.empty(0, 64, device="cuda"), "mxfp4")
    assert codes.shape == (0, 32) and scales.shape == (2, 0)
    X = torch.randn(100, 320, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scales = capi.mx_quantize(X, "mxfp8")
        back = capi.mx_dequantize(codes, scales, "mxfp8", torch.float32)
    X.normal_()
    graph.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c2, s2 = capi.mx_quantize(X, "mxfp8", stream=s)
    torch.cuda.synchronize()
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    assert torch.equal(back, capi.mx_dequantize(c2, s2, "mxfp8", torch.float32))


def test_large_offsets():
    """More than 2^31 values."""
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs 40 GB")
    X = torch.zeros(2, 600_001, 2048, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(5)
    X[1, -3:] = torch.randn(3, 2048, generator=gen).to(torch.bfloat16).cuda()
    codes, scales = capi.mx_quantize(X, "mxfp4")
    code, scale = _define(X[1, -3:], "mxfp4")
    assert torch.equal(_unpacked(codes[1, -3:], "mxfp4"), code) and torch.equal(scales[1, :, -3:].cpu(), scale)
    assert int(codes[:, :-3].count_nonzero()) == 0
    back = capi.mx_dequantize(codes, scales, "mxfp4")
    assert torch.equal(back[1, -3:].double().cpu(), _values(code, scale, "mxfp4"))


def test_refusals():
    X = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="fmt"):
        capi.mx_quantize(X, "fp4")
    with pytest.raises(ValueError, match="dtype"):
        capi.mx_quantize(X.half(), "mxfp4")
    with pytest.raises(ValueError, match="contiguous"):
        capi.mx_quantize(torch.zeros(64, 4, device="cuda").t(), "mxfp4")
    with pytest.raises(ValueError, match="rows, K"):
        capi.mx_quantize(X.flatten(), "mxfp4")
    with pytest.raises(ValueError, match="shape"):
        capi.mx_quantize(X, "mxfp4", codes=torch.zeros(4, 64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(capi.MoeError, match="multiple of 32"):
        capi.mx_quantize(torch.zeros(4, 48, device="cuda"), "mxfp8")
    with pytest.raises(capi.MoeError, match="aligned"):
        capi.mx_quantize(torch.zeros(65, device="cuda")[1:].view(2, 32), "mxfp8")
