"""moe_mx_grouped_forward against fp64 on the decoded operands.

Tolerance, derived before the first run: a product of two E2M1 values and two powers of two
is exact in fp32, so an element of n products is off by at most n * 2^-23 * sum |x w|
(whatever the order of the sum, rounding or truncating), then rounded once."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


def _offs(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32,
                        device="cuda")


def _operands(counts, N, K, before=0, behind=0, seed=41):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = before + sum(counts) + behind
    # block magnitudes that differ by powers of two, so that a scale in the wrong place shows
    def tensor(*shape):
        spread = torch.randint(-6, 7, shape[:-1] + (shape[-1] // 32,), generator=gen, device="cuda")
        return torch.randn(shape, generator=gen, device="cuda") * torch.exp2(spread.float()).repeat_interleave(32, -1)

    X, W = capi.mx_quantize(tensor(rows, K), "mxfp4"), capi.mx_quantize(tensor(len(counts), N, K), "mxfp4")
    return X, W, _offs(counts, before)


def _values(q):
    return capi.mx_dequantize(*q, "mxfp4", torch.float32).double()


def _check(got, X, W, offs):
    o = offs.tolist()
    x, w = _values(X), _values(W)
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        ref, mag = x[r] @ w[e].t(), x[r].abs() @ w[e].abs().t()
        bound = x.shape[1] * 2.0 ** -23 * mag
        bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound)
        off = (got[r].double() - ref).abs()
        assert bool((off <= bound).all()), (e, int((off > bound).sum()), float((off / (bound + 1e-300)).max()))


CASES = {
    "one_row": ([1], 64, 32, 0, 0),
    "tiny_sizes": ([3, 1], 8, 32, 0, 0),
    "odd": ([5, 0, 130, 17, 0, 64, 33], 200, 352, 0, 0),
    "spare": ([5, 0, 130, 17, 0, 64, 33], 72, 96, 7, 29),
    "all_empty": ([0, 0, 0], 64, 64, 0, 40),
    "first_empty": ([0, 256, 1], 256, 256, 0, 3),
    "tokens": ([1, 0, 0, 1, 0, 1, 1] + [0] * 50 + [2], 1408, 2048, 0, 0),
    "many_experts": ([(7 * i) % 41 for i in range(256)], 136, 192, 0, 1),
    "one_expert_large": ([1500], 1032, 1568, 0, 0),
    "wide": ([700, 900], 4104, 64, 0, 0),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", list(CASES))
def test_against_fp64(name, dtype):
    counts, N, K, before, behind = CASES[name]
    X, W, offs = _operands(counts, N, K, before, behind)
    rows = X[0].shape[0]
    out = torch.full((rows, N), -3.0, dtype=dtype, device="cuda")
    assert capi.mx_grouped_forward(*X, *W, offs, out=out) is out
    _check(out, X, W, offs)
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    own[before:before + sum(counts)] = True
    assert bool((out[~own] == -3.0).all()), "rows that no expert owns were written"
    again = capi.mx_grouped_forward(*X, *W, offs, out_dtype=dtype)
    assert torch.equal(again[own], out[own])


def test_every_code_and_scale_place():
    """One-hot rows: each output is one product, so every code, nibble, block and scale is seen alone."""
    K, N = 352, 72
    gen = torch.Generator().manual_seed(42)
    Wc = torch.randint(0, 256, (1, N, K // 2), generator=gen, dtype=torch.uint8).cuda()
    Ws = torch.randint(110, 140, (1, K // 32, N), generator=gen, dtype=torch.uint8).cuda()
    Xc = torch.zeros(K, K // 2, dtype=torch.uint8)
    for k in range(K):
        Xc[k, k // 2] = (1 + k % 15) << (4 * (k % 2))
    Xs = torch.randint(110, 140, (K // 32, K), generator=gen, dtype=torch.uint8).cuda()
    X, W = (Xc.cuda(), Xs), (Wc, Ws)
    got = capi.mx_grouped_forward(*X, *W, _offs([K]), out_dtype=torch.float32)
    assert torch.equal(got.double(), _values(X) @ _values(W)[0].t())


def test_non_finite_blocks_stay_in_their_rows():
    X, W, offs = _operands([40, 100, 3], 136, 320)
    clean = capi.mx_grouped_forward(*X, *W, offs)
    X[1][3, 17] = 255   # a block of row 17 (expert 0)
    X[1][9, 141] = 255  # the last block of a row of expert 2
    W[1][1, 4, 100] = 255
    got = capi.mx_grouped_forward(*X, *W, offs)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[17], nan[141], nan[40:140, 100] = True, True, True
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], clean[~nan])


def test_others_rows_do_not_reach_a_result():
    X, W, offs = _operands([20, 0, 45, 9], 72, 224, 3, 5)
    clean = capi.mx_grouped_forward(*X, *W, offs)
    X[1][:, :3] = X[1][:, 77:] = X[1][:, 23:68] = 255
    W[1][1] = 255
    got = capi.mx_grouped_forward(*X, *W, offs)
    assert torch.equal(got[3:23], clean[3:23]) and torch.equal(got[68:77], clean[68:77])
    assert bool(got[23:68].isnan().all())


@pytest.mark.parametrize("offs", [[0, 5, 3, 9], [-1, 2, 4, 9], [0, 2, 4, 11]])
def test_bad_offsets_write_nothing(offs):
    X, W, _ = _operands([4, 4, 2], 64, 64)
    out = torch.full((10, 64), 7.0, device="cuda")
    capi.mx_grouped_forward(*X, *W, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=out)
    assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK
    assert bool((out == 7.0).all())


def test_streams_graphs_and_no_rows():
    X, W, offs = _operands([50, 0, 77, 140], 264, 320)
    want = capi.mx_grouped_forward(*X, *W, offs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = capi.mx_grouped_forward(*X, *W, offs, stream=s)
    graph = torch.cuda.CUDAGraph()
    source = capi.mx_dequantize(*X, "mxfp4", torch.bfloat16)
    with torch.cuda.graph(graph):
        q = capi.mx_quantize(source, "mxfp4")
        y = capi.mx_grouped_forward(*q, *W, offs)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, other) and torch.equal(want, y)
    source.normal_()
    graph.replay()
    torch.cuda.synchronize()
    _check(y, q, W, offs)
    none = capi.mx_grouped_forward(X[0][:0], X[1][:, :0].contiguous(), *W, torch.zeros_like(offs))
    assert none.shape == (0, 264)


def test_refusals():
    X, W, offs = _operands([4, 4], 64, 64)
    with pytest.raises(ValueError, match="Xs"):
        capi.mx_grouped_forward(X[0], X[1].t().contiguous(), *W, offs)
    with pytest.raises(ValueError, match="uint8"):
        capi.mx_grouped_forward(X[0].char(), X[1], *W, offs)
    with pytest.raises(ValueError, match="offs"):
        capi.mx_grouped_forward(*X, *W, offs[:2])
    with pytest.raises(capi.MoeError, match="UNSUPPORTED"):
        capi.mx_grouped_forward(X[0][:, :24].contiguous(), X[1][:1], W[0][:, :, :24].contiguous(), W[1][:, :1].contiguous(), offs)


# rows and N multiples of 16, so that scales come by TMA: behind fills the rows up
ALIGNED = {
    "one_block": ([16], 16, 32, 0),
    "two_rows": ([1, 0, 1], 32, 64, 0),
    "ragged_starts": ([5, 0, 130, 17, 0, 64, 33], 208, 352, 3),
    "many_experts": ([(7 * i) % 41 for i in range(256)], 144, 192, 5),
    "more_than_a_chunk": ([1, 7, 200, 15, 193], 272, 2752, 0),
    "one_expert_large": ([1504], 1040, 1568, 0),
    "tokens": ([1, 0, 0, 1, 0, 1, 1] + [0] * 50 + [2], 1408, 2048, 0),
    "exact_tiles": ([192, 384, 192], 256, 512, 0),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", list(ALIGNED))
def test_aligned_sizes(name, dtype):
    """Against fp64, and bit for bit what the same rows give with one more behind them."""
    counts, N, K, before = ALIGNED[name]
    X, W, offs = _operands(counts, N, K, before, -(before + sum(counts)) % 16, seed=43)
    rows = X[0].shape[0]
    out = torch.full((rows, N), -3.0, dtype=dtype, device="cuda")
    capi.mx_grouped_forward(*X, *W, offs, out=out)
    _check(out, X, W, offs)
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    own[before:before + sum(counts)] = True
    assert bool((out[~own] == -3.0).all())
    more = torch.cat([X[0], X[0][:1]]), torch.cat([X[1], X[1][:, :1]], 1)
    assert torch.equal(capi.mx_grouped_forward(*more, *W, offs, out_dtype=dtype)[:rows][own], out[own])


def test_aligned_non_finite_blocks_stay_in_their_rows():
    X, W, offs = _operands([40, 100, 3], 144, 1056, 1, 16)
    clean = capi.mx_grouped_forward(*X, *W, offs)
    X[1][3, 18] = X[1][32, 142] = 255  # row 17 of expert 0; the last block of a row of expert 2
    X[1][:, 0] = X[1][:, 144:] = 255   # no expert's rows
    W[1][1, 4, 100] = 255
    got = capi.mx_grouped_forward(*X, *W, offs)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[18], nan[142], nan[41:141, 100] = True, True, True
    assert torch.equal(got[1:144].isnan(), nan[1:144])
    assert torch.equal(got[1:144][~nan[1:144]], clean[1:144][~nan[1:144]])
