"""The gated block's products (moe_grouped_gated_forward / _backward / _dgrad) against fp64.

Tolerances, derived before the first run.  A sum of n products of bf16 values is off by at most
d = n 2^-23 sum |a b| (tests/test_gpu_grouped.py).  The activation in fp32: exp to 2 + 1.173 |x| units
in the last place (2^-23), the addition, the quotient (2 units) and up to four products more, so
the sigmoid s(x) is off by e = (8 + 1.2 |x|) 2^-23 of itself at most.  x -> x s(a x) has slopes up to
1.1, clamps have slopes up to 1, so with a(g) = g' s(alpha g') and v = u' + beta
  H   1.1 d_g (|v| + d_u) + |a| d_u + e |a v|
  dG  d |D| + |dH| |v| (1 + |alpha g|) (2 e + 2^-21),  D = v s (1 + alpha g (1 - s))
  dU  d |a| + e |dH a|
(1 - s is off by e + 2^-24, and is multiplied by |alpha g|.)  Values under 2^-100 may be flushed by
the quotient.  Then one rounding: half a step of the value.
"""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

ALPHA, LIMIT, BETA = 1.702, 7.0, 1.0
BF = torch.bfloat16


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
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(BF)


def _offs(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32,
                        device="cuda")


def _own(rows, offs):
    at = torch.arange(rows, device="cuda")
    return (at >= offs[0]) & (at < offs[-1])


def _product(A, W, offs, across):
    """fp64 A[r] W[e]^T (across) or A[r] W[e], the bound of its fp32 sum, zeros in rows of no expert."""
    o = offs.tolist()
    cols = W.shape[1] if across else W.shape[2]
    ref = torch.zeros(A.shape[0], cols, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        w = W[e].double().t() if across else W[e].double()
        ref[r] = A[r].double() @ w
        mag[r] = A[r].double().abs() @ w.abs()
    return ref, A.shape[1] * 2.0 ** -23 * mag


def _parts(g, u, act):
    """a(g), v, s, |alpha g|, and which gradients pass, in fp64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, u, s, g.abs(), torch.ones_like(g), torch.ones_like(u)
    gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    s = torch.sigmoid(ALPHA * gc)
    return gc * s, uc + BETA, s, (ALPHA * gc).abs(), (g <= LIMIT).double(), (u.abs() <= LIMIT).double()


def _near(got, ref, bound, own):
    bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound) + 2.0 ** -100
    bad = ((got.double() - ref).abs() > bound) | ~torch.isfinite(got)
    assert not bool(bad[own].any()), (int(bad[own].sum()), float(((got.double() - ref).abs() / bound)[own].max()))


CASES = {  # counts, I, K, rows before the first expert, rows behind the last
    "one_row": ([1], 64, 64, 0, 0),
    "tiny_sizes": ([3, 1], 8, 8, 0, 0),
    "odd": ([5, 0, 130, 17, 0, 64, 33], 200, 328, 0, 0),
    "spare": ([5, 0, 130, 17, 0, 64, 33], 72, 136, 7, 29),
    "all_empty": ([0, 0, 0], 64, 72, 0, 40),
    "last_empty": ([129, 255, 0], 264, 520, 0, 0),
    "first_empty": ([0, 256, 1], 136, 256, 0, 3),
    "tokens": ([1, 0, 0, 1, 0, 1, 1] + [0] * 50 + [2], 1408, 2048, 0, 0),
    "many_experts": ([(7 * i) % 41 for i in range(256)], 136, 192, 0, 1),
    "one_expert_large": ([1500], 1024, 1544, 0, 0),
    "tails": ([15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129], 328, 96, 0, 0),
    "long": ([40, 3], 4168, 16456, 0, 0),
}


@pytest.mark.parametrize("act", ["silu", "swigluoai"])
@pytest.mark.parametrize("name", list(CASES))
def test_forward(name, act):
    counts, I, K, before, behind = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(11)
    E, rows = len(counts), before + sum(counts) + behind
    std = 3 / K ** 0.5  # the clamped activation's limit is passed now and then
    X, Wg, Wu = _bf16(gen, rows, K), _bf16(gen, E, I, K, std=std), _bf16(gen, E, I, K, std=std)
    offs = _offs(counts, before)
    outs = [torch.full((rows, I), -3.0, dtype=BF, device="cuda") for _ in range(3)]
    H, G, U = capi.grouped_gated_forward(X, Wg, Wu, offs, act=act, out=outs[0], save=(outs[1], outs[2]))
    assert H is outs[0] and G is outs[1] and U is outs[2]
    own = _own(rows, offs)
    for t in outs:
        assert bool((t[~own] == -3.0).all()), "rows that no expert owns were written"
    (g, dg), (u, du) = _product(X, Wg, offs, True), _product(X, Wu, offs, True)
    _near(G, g, dg, own)
    _near(U, u, du, own)
    a, v, _, x, _, _ = _parts(g, u, act)
    _near(H, a * v, 1.1 * dg * (v.abs() + du) + a.abs() * du + (8 + 1.2 * x) * 2.0 ** -23 * (a * v).abs(), own)
    alone = capi.grouped_gated_forward(X, Wg, Wu, offs, act=act)
    assert torch.equal(alone[own], H[own])
    again = capi.grouped_gated_forward(X, Wg, Wu, offs, act=act, save=True)
    assert all(torch.equal(p[own], q[own]) for p, q in zip(again, outs))


@pytest.mark.parametrize("act", ["silu", "swigluoai"])
@pytest.mark.parametrize("name", list(CASES))
def test_backward(name, act):
    counts, I, K, before, behind = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(12)
    E, rows = len(counts), before + sum(counts) + behind
    dY, Wd = _bf16(gen, rows, K), _bf16(gen, E, K, I, std=1 / K ** 0.5)
    G, U = _bf16(gen, rows, I, std=3), _bf16(gen, rows, I, std=3)
    if rows > 1:  # at the limits, and far from zero
        G[::2, 0], U[::2, 1], U[::2, 2] = LIMIT, LIMIT, -LIMIT
        G[::2, 3], G[::2, 4], U[::2, 5] = -120.0, 60.0, 1e4
    offs = _offs(counts, before)
    outs = [torch.full((rows, I), -3.0, dtype=BF, device="cuda") for _ in range(2)]
    dG, dU = capi.grouped_gated_backward(dY, Wd, G, U, offs, act=act, out=outs)
    assert dG is outs[0] and dU is outs[1]
    own = _own(rows, offs)
    for t in outs:
        assert bool((t[~own] == -3.0).all()), "rows that no expert owns were written"
    dh, d = _product(dY, Wd, offs, False)
    a, v, s, x, pass_g, pass_u = _parts(G.double(), U.double(), act)
    sign = torch.sign(G.double())
    D = v * s * (1 + sign * x * (1 - s)) * pass_g
    e = (8 + 1.2 * x) * 2.0 ** -23
    _near(dG, dh * D, d * D.abs() + dh.abs() * v.abs() * (1 + x) * (2 * e + 2.0 ** -21), own)
    _near(dU, dh * a * pass_u, d * a.abs() + e * (dh * a).abs(), own)
    again = capi.grouped_gated_backward(dY, Wd, G, U, offs, act=act)
    assert all(torch.equal(p[own], q[own]) for p, q in zip(again, outs))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("name", list(CASES))
def test_dgrad(name, dtype):
    counts, I, K, before, behind = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(13)
    E, rows = len(counts), before + sum(counts) + behind
    dG, dU = _bf16(gen, rows, I), _bf16(gen, rows, I)
    Wg, Wu = _bf16(gen, E, I, K, std=0.05), _bf16(gen, E, I, K, std=0.05)
    offs = _offs(counts, before)
    out = torch.full((rows, K), -3.0, dtype=dtype, device="cuda")
    assert capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out=out) is out
    own = _own(rows, offs)
    assert bool((out[~own] == -3.0).all()), "rows that no expert owns were written"
    (a, da), (b, db) = _product(dG, Wg, offs, False), _product(dU, Wu, offs, False)
    _near(out, a + b, 2 * (da + db), own)  # one sum of twice as many products
    again = capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out_dtype=dtype)
    assert again.dtype == dtype and torch.equal(again[own], out[own])


@pytest.mark.parametrize("I", [256, 264, 512, 768, 1400, 8200])
@pytest.mark.parametrize("counts", [[1, 0, 37, 64], [300, 1, 513]])
def test_dgrad_fp32_sums_are_exact_ones(counts, I):
    # Operands of one sign, where truncation shows most.  A segment's 32 additions lose up to 2^-23 of
    # its sum each, the sums of segments 2^-24 of the whole each: 2^-18 + segments 2^-24.
    K, rows = 328, sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(29)
    dG, dU = _bf16(gen, rows, I).abs(), _bf16(gen, rows, I).abs()
    Wg, Wu = _bf16(gen, len(counts), I, K).abs(), _bf16(gen, len(counts), I, K).abs()
    offs = _offs(counts)
    out = capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out_dtype=torch.float32)
    ref = _product(dG, Wg, offs, False)[0] + _product(dU, Wu, offs, False)[0]
    segments = -(-2 * (I + 63) // 512)
    _near(out, ref, (2.0 ** -18 + segments * 2.0 ** -24) * ref, _own(rows, offs))


@pytest.mark.parametrize("act", ["silu", "swigluoai"])
def test_gradients_against_differences(act):
    """The backward chain against central differences of the fp64 block, in random directions.

    Half the difference over a step t of 2^-10 is off by t^2 / 6 of a third derivative; what the
    call rounds (G, U, dG, dU, dX to bf16) is compared as vectors: 2^-8 of each gradient's norm
    from each of at most three roundings, against which t^2 is nothing."""
    gen = torch.Generator(device="cuda").manual_seed(14)
    counts, I, K = [37, 0, 64, 5], 72, 88
    E, rows = len(counts), sum(counts)
    X, Wg, Wu = _bf16(gen, rows, K), _bf16(gen, E, I, K, std=0.2), _bf16(gen, E, I, K, std=0.2)
    Wd, dY = _bf16(gen, E, K, I, std=0.2), _bf16(gen, rows, K)
    offs = _offs(counts)
    H, G, U = capi.grouped_gated_forward(X, Wg, Wu, offs, act=act, save=True)
    dG, dU = capi.grouped_gated_backward(dY, Wd, G, U, offs, act=act)
    got = {"X": capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out_dtype=torch.float32),
           "Wg": capi.grouped_wgrad(dG, X, offs), "Wu": capi.grouped_wgrad(dU, X, offs), "Wd": capi.grouped_wgrad(dY, H, offs)}

    def loss(x, wg, wu, wd):
        g, u = _product(x, wg, offs, True)[0], _product(x, wu, offs, True)[0]
        a, v, *_ = _parts(g, u, act)
        return (dY.double() * _product(a * v, wd, offs, True)[0]).sum()

    at = {"X": X.double(), "Wg": Wg.double(), "Wu": Wu.double(), "Wd": Wd.double()}
    t = 2.0 ** -10
    for name, grad in got.items():
        # along the gradient itself: the difference is its norm, or the call's gradient is not that
        direction = grad.double() / grad.double().norm()
        ends = [loss(*[p + sign * t * direction if n == name else p for n, p in at.items()]) for sign in (1, -1)]
        slope = float(ends[0] - ends[1]) / (2 * t)
        norm = float(grad.double().norm())
        assert abs(slope - norm) <= 3 * 2.0 ** -8 * norm, (name, slope, norm)


def test_other_rows_and_experts_stay_clean():
    """A NaN or an infinity reaches the rows and columns whose sums hold it and no others."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    counts, I, K = [33, 31, 70], 72, 72
    E, rows = 3, sum(counts) + 9
    offs = _offs(counts)
    X, Wg, Wu = _bf16(gen, rows, K), _bf16(gen, E, I, K, std=0.1), _bf16(gen, E, I, K, std=0.1)
    clean = capi.grouped_gated_forward(X, Wg, Wu, offs)
    X2, Wg2 = X.clone(), Wg.clone()
    X2[sum(counts):] = float("nan")  # rows of no expert
    X2[40] = float("inf")
    Wg2[0, 5, 3] = float("nan")
    H = capi.grouped_gated_forward(X2, Wg2, Wu, offs)
    assert bool(torch.isnan(H[:33, 5]).all())
    assert not bool(torch.isfinite(H[40]).any())
    keep = torch.ones(rows, I, dtype=torch.bool, device="cuda")
    keep[sum(counts):], keep[40], keep[:33, 5] = False, False, False
    assert torch.equal(H[keep], clean[keep])
    # the clamped activation passes a NaN on
    H = capi.grouped_gated_forward(X2, Wg2, Wu, offs, act="swigluoai")
    assert bool(torch.isnan(H[:33, 5]).all())
    dG, dU = _bf16(gen, rows, I), _bf16(gen, rows, I)
    clean = capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs)
    dU[sum(counts):], dG[7] = float("inf"), float("nan")
    dX = capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs)
    assert bool(torch.isnan(dX[7]).all())
    keep = torch.arange(rows, device="cuda") < sum(counts)
    keep[7] = False
    assert torch.equal(dX[keep], clean[keep])


def test_projections_next_to_each_other():
    """Gate and up as halves of one tensor; sizes that end inside a box."""
    gen = torch.Generator(device="cuda").manual_seed(16)
    counts, I, K = [20, 44], 8, 40
    both = _bf16(gen, 2, 2, I, K)
    X, offs = _bf16(gen, 64, K), _offs(counts)
    H = capi.grouped_gated_forward(X, both[1], both[0], offs)
    assert torch.equal(H, capi.grouped_gated_forward(X, both[1].clone(), both[0].clone(), offs))
    same = capi.grouped_gated_forward(X, both[0], both[0], offs)  # the same tensor twice
    assert torch.equal(same, capi.grouped_gated_forward(X, both[0], both[0].clone(), offs))


def test_bad_offsets_write_nothing():
    X, W = torch.ones(16, 64, dtype=BF, device="cuda"), torch.ones(2, 64, 64, dtype=BF, device="cuda")
    for bad in ([0, 9, 17], [0, 8, 4], [-1, 4, 16]):
        offs = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out = torch.full((16, 64), -3.0, dtype=BF, device="cuda")
        out2 = out.clone()
        capi.grouped_gated_forward(X, W, W.clone(), offs, out=out)
        assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK and bool((out == -3.0).all())
        capi.grouped_gated_backward(X, W, X.clone(), X.clone(), offs, out=(out, out2))
        assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK and bool((out == -3.0).all()) and bool((out2 == -3.0).all())
        capi.grouped_gated_dgrad(X, X.clone(), W, W.clone(), offs, out=out)
        assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK and bool((out == -3.0).all())


def test_captured_and_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(17)
    counts, I, K = [100, 0, 29], 136, 264
    rows, offs = 129, _offs(counts)
    X, Wg, Wu = _bf16(gen, rows, K), _bf16(gen, 3, I, K, std=0.1), _bf16(gen, 3, I, K, std=0.1)
    Wd, dY = _bf16(gen, 3, K, I, std=0.1), _bf16(gen, rows, K)

    def step(stream=None):
        H, G, U = capi.grouped_gated_forward(X, Wg, Wu, offs, save=True, stream=stream)
        dG, dU = capi.grouped_gated_backward(dY, Wd, G, U, offs, stream=stream)
        return H, G, U, dG, dU, capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, stream=stream)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    X.copy_(_bf16(gen, rows, K))
    dY.copy_(_bf16(gen, rows, K))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_wait_bound_of_zero_gives_up():
    lib = capi.load()
    X, W = torch.ones(64, 64, dtype=BF, device="cuda"), torch.ones(1, 64, 64, dtype=BF, device="cuda")
    offs = _offs([64])
    try:
        assert lib.moe_operators_wait_limit(0) == capi.MOE_OK
        capi.grouped_gated_forward(X, W, W.clone(), offs)
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
        capi.grouped_gated_backward(X, W, X.clone(), X.clone(), offs)
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
        capi.grouped_gated_dgrad(X, X.clone(), W, W.clone(), offs)
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
    finally:
        assert lib.moe_operators_wait_limit(-1) == capi.MOE_OK
    got = capi.grouped_gated_dgrad(X, X.clone(), W, W.clone(), offs)
    assert bool((got == 128.0).all())


def test_python_refusals():
    X, W = torch.zeros(16, 64, dtype=BF, device="cuda"), torch.zeros(2, 32, 64, dtype=BF, device="cuda")
    offs = _offs([8, 8])
    for bad in (dict(Wu=W[:1]), dict(Wu=W.float()), dict(X=X.float()), dict(X=X[:, :32]), dict(offs=offs[:2]), dict(offs=offs.long()),
                dict(act="gelu"), dict(out=X), dict(save=(X, X)), dict(save=(torch.zeros(16, 32, dtype=BF, device="cuda"),)),
                dict(Wu=W.cpu())):
        args = {"X": X, "Wg": W, "Wu": W.clone(), "offs": offs, **bad}
        with pytest.raises(ValueError):
            capi.grouped_gated_forward(args.pop("X"), args.pop("Wg"), args.pop("Wu"), args.pop("offs"), **args)
    H = torch.zeros(16, 32, dtype=BF, device="cuda")
    with pytest.raises(capi.MoeError):
        capi.grouped_gated_forward(X, W, W.clone(), offs, out=H, save=(H, torch.zeros_like(H)))
    with pytest.raises(capi.MoeError):
        capi.grouped_gated_forward(X, W, W.clone(), offs, act="swigluoai", limit=float("nan"))
