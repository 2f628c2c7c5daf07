"""The grouped products (moe_grouped_forward / _dgrad / _wgrad) against fp64.

Tolerance of an element, derived before the first run: every product of two bf16 values
is exact in fp32, and a sum of n of them in fp32 is off by at most n * 2^-23 * sum |a b|
whatever the order and whether each addition rounds or truncates; the result is rounded
once to the output type (half a step, eps / 2 of the value).
"""

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


def _bf16(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _offs(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32,
                        device="cuda")


def _reference(op, A, B, offs, shape):
    """fp64 result and, per element, the sum of the products' magnitudes and their number."""
    o = offs.tolist()
    ref = torch.zeros(shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    num = torch.zeros([shape[0]] + [1] * (len(shape) - 1), dtype=torch.float64, device="cuda")
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        if op == "wgrad":
            a, b, at = A[r].double().t(), B[r].double(), e
        else:
            w = B[e].double()
            a, b, at = A[r].double(), (w.t() if op == "forward" else w), r
        ref[at] = a @ b
        mag[at] = a.abs() @ b.abs()
        num[at] = a.shape[1]
    return ref, mag, num


def _check(got, ref, mag, num):
    half = torch.finfo(got.dtype).eps / 2
    # the fp32 sum, then one rounding of it
    bound = num * 2.0 ** -23 * mag
    bound = bound + half * (ref.abs() + bound)
    bad = (got.double() - ref).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - ref).abs() / (bound + 1e-300)).max()))


def _call(op, A, B, offs, **kw):
    return {"forward": capi.grouped_forward, "dgrad": capi.grouped_dgrad, "wgrad": capi.grouped_wgrad}[op](A, B, offs, **kw)


def _inputs(op, rows, E, N, K, gen):
    X, dY, W = _bf16(gen, rows, K), _bf16(gen, rows, N), _bf16(gen, E, N, K, std=0.05)
    return {"forward": (X, W), "dgrad": (dY, W), "wgrad": (dY, X)}[op]


def _shape(op, rows, E, N, K):
    return {"forward": (rows, N), "dgrad": (rows, K), "wgrad": (E, N, K)}[op]


CASES = {  # counts, N, K, rows before the first expert, rows behind the last
    "one_row": ([1], 64, 64, 0, 0),
    "tiny_sizes": ([3, 1], 8, 8, 0, 0),
    "odd": ([5, 0, 130, 17, 0, 64, 33], 200, 328, 0, 0),
    "spare": ([5, 0, 130, 17, 0, 64, 33], 72, 136, 7, 29),
    "all_empty": ([0, 0, 0], 64, 72, 0, 40),
    "last_empty": ([129, 255, 0], 264, 520, 0, 0),
    "first_empty": ([0, 256, 1], 256, 256, 0, 3),
    "tokens": ([1, 0, 0, 1, 0, 1, 1] + [0] * 50 + [2], 1408, 2048, 0, 0),
    "many_experts": ([(7 * i) % 41 for i in range(256)], 136, 192, 0, 1),
    "one_expert_large": ([1500], 1024, 1544, 0, 0),
    "tails": ([15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129], 328, 96, 0, 0),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("name", list(CASES))
def test_against_fp64(name, op, dtype):
    counts, N, K, before, behind = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(5)
    E, rows = len(counts), before + sum(counts) + behind
    A, B = _inputs(op, rows, E, N, K, gen)
    offs = _offs(counts, before)
    out = torch.full(_shape(op, rows, E, N, K), -3.0, dtype=dtype, device="cuda")
    got = _call(op, A, B, offs, out=out)
    assert got is out
    ref, mag, num = _reference(op, A, B, offs, out.shape)
    if op != "wgrad":
        own = torch.zeros(rows, dtype=torch.bool, device="cuda")
        own[before:before + sum(counts)] = True
        assert bool((got[~own] == -3.0).all()), "rows that no expert owns were written"
        got, ref, mag, num = got[own], ref[own], mag[own], num[own]
    _check(got, ref, mag, num)
    again = _call(op, A, B, offs, out_dtype=dtype)
    assert again.dtype == dtype
    if op == "wgrad":
        assert torch.equal(again, out)
    else:
        assert torch.equal(again[own], got)


@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_rows_of_others_do_not_reach_a_result(op):
    """Infinities and NaN in another expert's rows, behind the last one, and in an unused expert's weights."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    counts, N, K = [20, 0, 45, 9], 72, 200
    offs = _offs(counts, 3)
    rows = 3 + sum(counts) + 5
    A, W = _inputs(op, rows, 4, N, K, gen)
    clean = _call(op, A, W, offs)
    A[:3], A[3 + sum(counts):] = float("nan"), float("inf")
    A[23:68] = float("nan")  # expert 2
    W[1] = float("inf")
    got = _call(op, A, W, offs)
    assert torch.equal(got[3:23], clean[3:23]) and torch.equal(got[68:77], clean[68:77])
    assert bool(got[23:68].isnan().all())


def test_wgrad_reads_only_its_rows():
    """The rows past an expert's end, inside its last k-block, may hold anything."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    counts = [9, 70, 16, 1]
    offs = _offs(counts, 2)
    dY, X = _inputs("wgrad", 2 + sum(counts) + 6, 4, 96, 136, gen)
    clean = capi.grouped_wgrad(dY, X, offs)
    for t, v in ((dY, float("nan")), (X, float("inf"))):
        t[:2] = t[2 + sum(counts):] = v
        t[11:81] = v  # expert 1
    got = capi.grouped_wgrad(dY, X, offs)
    for e in (0, 2, 3):
        assert torch.equal(got[e], clean[e]), e
    assert bool(got[1].isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad_accumulates(dtype):
    gen = torch.Generator(device="cuda").manual_seed(8)
    counts, N, K = [9, 0, 70, 131], 104, 264
    offs = _offs(counts)
    dY, X = _inputs("wgrad", sum(counts), 4, N, K, gen)
    base = torch.randn(4, N, K, generator=gen, device="cuda").to(dtype)
    out = base.clone()
    assert capi.grouped_wgrad(dY, X, offs, out=out, accumulate=True) is out
    ref, mag, num = _reference("wgrad", dY, X, offs, out.shape)
    assert torch.equal(out[1], base[1])
    # one more fp32 addition, rounded to nearest: 2^-24 of the sum
    total = ref + base.double()
    bound = num * 2.0 ** -23 * mag
    bound = bound + 2.0 ** -24 * (total.abs() + bound)
    bound = bound + torch.finfo(dtype).eps / 2 * (total.abs() + bound)
    assert bool(((out.double() - total).abs() <= bound).all())


def test_no_rows():
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(3, 72, 64, dtype=torch.bfloat16, device="cuda")
    assert capi.grouped_forward(X, W, offs).shape == (0, 72)
    dY = torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
    assert capi.grouped_dgrad(dY, W, offs).shape == (0, 64)
    out = torch.full((3, 72, 64), 2.0, device="cuda")
    assert bool((capi.grouped_wgrad(dY, X, offs, out=out, accumulate=True) == 2).all())
    assert bool((capi.grouped_wgrad(dY, X, offs, out=out) == 0).all())


@pytest.mark.parametrize("offs", [[0, 5, 3, 9], [-1, 2, 4, 9], [0, 2, 4, 11]])
@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
def test_bad_offsets_write_nothing(op, offs):
    gen = torch.Generator(device="cuda").manual_seed(9)
    A, B = _inputs(op, 10, 3, 64, 72, gen)
    out = torch.full(_shape(op, 10, 3, 64, 72), 7.0, device="cuda")
    _call(op, A, B, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=out)
    assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK
    assert "offsets" in capi.load().moe_last_error().decode()
    assert bool((out == 7.0).all())


def test_gradients_against_differences():
    """sum(Y * G) by X and by W: the gradients are exact derivatives of a function linear in
    each, so a difference quotient with any step is off by rounding alone."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    counts, N, K = [6, 0, 11], 24, 40
    offs = _offs(counts)
    X, W, G = _bf16(gen, 17, K), _bf16(gen, 3, N, K), _bf16(gen, 17, N)
    dX = capi.grouped_dgrad(G, W, offs, out_dtype=torch.float32)
    dW = capi.grouped_wgrad(G, X, offs)

    def loss(X, W):
        return float((capi.grouped_forward(X, W, offs, out_dtype=torch.float32).double() * G.double()).sum())

    # each loss is off by at most K 2^-23 sum |G| |W| |X| (the products' sums; the rest is fp64)
    mag = float((capi.grouped_forward(X.abs(), W.abs(), offs, out_dtype=torch.float32).double() * G.double().abs()).sum())
    for i, j in ((0, 0), (5, 39), (6, 7), (16, 20)):
        at = X[i, j].item()
        X[i, j] = 64.0
        high = loss(X, W)
        X[i, j] = -64.0
        low = loss(X, W)
        X[i, j] = at
        slack = 2 * (K + 1) * 2.0 ** -23 * (mag + 64 * float(G.double().abs()[i] @ W.double().abs()[0 if i < 6 else 2][:, j])) / 128
        assert abs((high - low) / 128 - float(dX[i, j])) <= slack + 2.0 ** -22 * N * float(dX.abs().max())
    for e, n, k in ((0, 0, 0), (2, 23, 39), (2, 4, 9), (1, 3, 3)):
        at = W[e, n, k].item()
        W[e, n, k] = 64.0
        high = loss(X, W)
        W[e, n, k] = -64.0
        low = loss(X, W)
        W[e, n, k] = at
        slack = 2 * (K + 1) * 2.0 ** -23 * (mag + 64 * float(G.double().abs()[:, n] @ X.double().abs()[:, k])) / 128
        assert abs((high - low) / 128 - float(dW[e, n, k])) <= slack + 2.0 ** -22 * 17 * float(dW.abs().max())


def test_streams_and_graphs():
    """Two streams at once, and a captured call replayed on new contents of the same tensors."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    counts, N, K = [40, 0, 90, 3], 264, 320
    offs = _offs(counts)
    X, W = _inputs("forward", 133, 4, N, K, gen)
    dY = _bf16(gen, 133, N)
    want = capi.grouped_forward(X, W, offs), capi.grouped_dgrad(dY, W, offs), capi.grouped_wgrad(dY, X, offs)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a = capi.grouped_forward(X, W, offs, stream=s1)
        b = capi.grouped_dgrad(dY, W, offs, stream=s2)
        c = capi.grouped_wgrad(dY, X, offs, stream=s1)
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = capi.grouped_forward(X, W, offs)
        dx = capi.grouped_dgrad(y, W, offs)
        dw = capi.grouped_wgrad(y, X, offs)
    X.copy_(_bf16(gen, *X.shape))
    offs.copy_(_offs([10, 60, 0, 63]))
    graph.replay()
    torch.cuda.synchronize()
    y2 = capi.grouped_forward(X, W, offs)
    assert torch.equal(y, y2) and torch.equal(dx, capi.grouped_dgrad(y2, W, offs))
    assert torch.equal(dw, capi.grouped_wgrad(y2, X, offs))


def test_long_offsets():
    """More than 2^31 bytes and 2^31 elements behind one pointer."""
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs 40 GB")
    rows, N, K = 2_200_000, 8, 1024  # X and the dgrad's result: 2.25e9 elements
    gen = torch.Generator(device="cuda").manual_seed(12)
    W = _bf16(gen, 2, N, K)
    dY = _bf16(gen, rows, N)
    cut = 2_150_001
    offs = torch.tensor([0, cut, rows], dtype=torch.int32, device="cuda")
    dX = capi.grouped_dgrad(dY, W, offs)
    for r in (0, cut - 1, cut, rows - 1):
        ref, mag, num = _reference("dgrad", dY[r:r + 1], W[int(r >= cut):][:1], _offs([1]), (1, K))
        _check(dX[r:r + 1], ref, mag, num)
    Y = capi.grouped_forward(dX, W, offs)
    tail = slice(rows - 64, rows)
    ref, mag, num = _reference("forward", dX[tail], W[1:], _offs([64]), (64, N))
    _check(Y[tail], ref, mag, num)


def test_refuses_what_it_cannot_take():
    lib = capi.load()
    X = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(2, 72, 64, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, 8, 16], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="bfloat16"):
        capi.grouped_forward(X.float(), W, offs)
    with pytest.raises(ValueError, match="shape"):
        capi.grouped_forward(X[:, :32].contiguous(), W, offs)
    with pytest.raises(ValueError, match="contiguous"):
        capi.grouped_forward(X, W.transpose(1, 2).contiguous().transpose(1, 2), offs)
    with pytest.raises(ValueError, match="int32"):
        capi.grouped_forward(X, W, offs.long())
    with pytest.raises(ValueError, match="shape"):
        capi.grouped_dgrad(X, W, offs)
    with pytest.raises(ValueError, match="device"):
        capi.grouped_forward(X, W, offs.cpu())
    with pytest.raises(ValueError, match="out"):
        capi.grouped_wgrad(X, X, offs, accumulate=True)
    with pytest.raises(ValueError, match="shape"):
        capi.grouped_wgrad(X, X[:8].contiguous(), offs)
    with pytest.raises(capi.MoeError, match="aligned"):
        capi.grouped_forward(torch.zeros(16 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(16, 64), W, offs)
    with pytest.raises(capi.MoeError, match="UNSUPPORTED"):
        capi.grouped_forward(X[:, :60].contiguous(), W[:, :, :60].contiguous(), offs)
    assert lib.moe_operators_status() == capi.MOE_OK


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
def test_long_sums_keep_their_precision(op):
    """Sums of positive products, the worst case of additions that truncate.  fp32 outputs are
    summed in segments of 4096: a segment's 256 additions of 16 products lose at most 2^-23 of the
    running sum each, on average half of the last one's (256 / 2 * 2^-23 = 2^-16 at most), those
    of the segments half a step each; 2^-15 leaves a factor of almost two for the order in the 16."""
    gen = torch.Generator(device="cuda").manual_seed(51)
    long, N, counts = 40_016, 136, [40_016, 0, 4096, 8200] if op == "wgrad" else [70, 0, 33, 1]
    if op == "wgrad":
        A, B = _bf16(gen, sum(counts), N).abs(), _bf16(gen, sum(counts), 264).abs()
    else:
        A = _bf16(gen, sum(counts), long).abs()
        B = _bf16(gen, *((4, N, long) if op == "forward" else (4, long, N))).abs()
    offs = _offs(counts)
    got = _call(op, A, B, offs, out_dtype=torch.float32)
    ref, mag, num = _reference(op, A, B, offs, tuple(got.shape))
    assert bool(((got.double() - ref).abs() <= 2.0 ** -15 * ref).all())
    again = torch.zeros_like(got)
    _call(op, A, B, offs, out=again)
    assert torch.equal(again, got)
    if op == "wgrad":  # added to what is there: one more rounding of fp32 sums twice as large
        _call(op, A, B, offs, out=again, accumulate=True)
        assert bool(((again.double() - 2 * ref).abs() <= 2.0 ** -15 * 2 * ref).all())


LENGTHS = [1, 15, 16, 17, 63, 64, 65, 79, 127, 128, 129, 143, 191, 192, 193, 255, 256, 257, 999, 0]


@pytest.mark.parametrize("rows", [64, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_sums_of_every_length(rows, dtype):
    """Sums that end anywhere in a stage, for tiles of few rows and of many; the rows around an
    expert's hold NaN in turn, which its own sum may not meet."""
    gen = torch.Generator(device="cuda").manual_seed(52)
    dY, X, offs = _bf16(gen, sum(LENGTHS), rows), _bf16(gen, sum(LENGTHS), 136), _offs(LENGTHS)
    ref, mag, num = _reference("wgrad", dY, X, offs, (len(LENGTHS), rows, 136))
    for odd in (0, 1):
        a, b = dY.clone(), X.clone()
        for e in range(odd, len(LENGTHS), 2):
            a[offs[e]:offs[e + 1]] = b[offs[e]:offs[e + 1]] = float("nan")
        mine = [e for e in range(1 - odd, len(LENGTHS), 2)]
        _check(_call("wgrad", a, b, offs, out_dtype=dtype)[mine], ref[mine], mag[mine], num[mine])


@pytest.mark.parametrize("counts", [[1, 0, 33, 2], [100, 0, 120, 3], [300, 500]])
@pytest.mark.parametrize("length", [8, 56, 64, 72, 120, 128, 136, 192, 200, 1000])
@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_sums_of_every_length(op, length, counts):
    gen = torch.Generator(device="cuda").manual_seed(53)
    A = _bf16(gen, sum(counts), length)
    B = _bf16(gen, *((len(counts), 264, length) if op == "forward" else (len(counts), length, 264)))
    got = _call(op, A, B, _offs(counts), out_dtype=torch.float32)
    _check(got, *_reference(op, A, B, _offs(counts), tuple(got.shape)))


@pytest.mark.parametrize("accumulate", [False, True])
def test_long_sum_among_many_experts(accumulate):
    """One expert's sum takes three segments, in tiles of full height; the others' take one.
    Tolerance as in test_long_sums_keep_their_precision."""
    gen = torch.Generator(device="cuda").manual_seed(54)
    counts = [3] * 20 + [8209] + [0, 70] * 10
    dY, X, offs = _bf16(gen, sum(counts), 256).abs(), _bf16(gen, sum(counts), 264).abs(), _offs(counts)
    ref, _, _ = _reference("wgrad", dY, X, offs, (len(counts), 256, 264))
    out = torch.ones_like(ref, dtype=torch.float32)
    _call("wgrad", dY, X, offs, out=out, accumulate=accumulate)
    ref = ref + (1.0 if accumulate else 0.0)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -15 * ref).all())
