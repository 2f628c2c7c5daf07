"""Sizes that do not fit the C ABI's int are refused, not cut to their lower 32 bits."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu
LONG = (1 << 32) + 64  # 64 as an int


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()
    if torch.cuda.get_device_properties(0).total_memory < 200e9:
        pytest.skip("needs 200 GB")
    yield
    torch.cuda.empty_cache()


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("shape", [(1, LONG), (1, 1, LONG)])
def test_quantise(shape, fmt):
    with pytest.raises(ValueError, match="2\\^31"):
        capi.mx_quantize(_empty(*shape), fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_dequantise(fmt):
    codes = _empty(1, LONG // 2 if fmt == "mxfp4" else LONG, dtype=torch.uint8)
    with pytest.raises(ValueError, match="2\\^31"):
        capi.mx_dequantize(codes, _empty(LONG // 32, 1, dtype=torch.uint8), fmt)


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
def test_products(op):
    offs = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    rows, W = _empty(LONG, 8), _empty(1, 8, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        if op == "wgrad":
            capi.grouped_wgrad(rows, rows, offs)
        else:
            getattr(capi, f"grouped_{op}")(rows, W, offs)


def test_mxfp4_product():
    offs = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        capi.mx_grouped_forward(_empty(LONG, 16, dtype=torch.uint8), _empty(1, LONG, dtype=torch.uint8),
                                _empty(1, 8, 16, dtype=torch.uint8), _empty(1, 1, 8, dtype=torch.uint8), offs)
