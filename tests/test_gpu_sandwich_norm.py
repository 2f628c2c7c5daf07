"""The norms around a block and their gradients (moe_sandwich_norm, _backward) against fp64.

Tolerances, derived before the first run, u = 2^-24.  A row's sum takes at most 48 additions in a
chain (16 values of a thread, 5 steps over a warp, 16 warps, and 11 to spare), so a sum of squares is
off by 48 u of itself and 1 / sqrt(mean + eps) by r = 32 u (24 u, and the quotient, the product, the
sum and the root).  Sums over T rows: (T + 40) u of the sum of magnitudes.  With d(.) for the error:
  X'  d = |g P| (r + 6 u) + 2 u (|a X| + |g P|)
  N   |w rx| (d(X') + |X'| (r + 6 u + |d(X')| / |X'|, as norms of the row))
  m = mean(dN w xh)   48 u mean|dN w xh| + |m| (r + 6 u)
  T   rx (|xh| d(m) + (|dN w| + |xh m|) (r + 8 u)) + 4 u (|dX'| + rx (|dN w| + |xh m|))
  dF  rf (|g w| d(T) + |fh| d(mf) + (|T g w| + |fh mf|) (r + 8 u)),
      d(mf) = mean(d(T) |g w fh| + |T g w fh| (r + 54 u))
  dw_pre   sum |dN xh| (r + 2 u + (T + 40) u); dw_post and dg likewise, with d(T) times the other factor.
1 % on top for products of errors, and one rounding, half a step of the value.
"""

import itertools

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
R = 32 * U
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


def _inputs(T, H, x_type, f_type, gate, kind, seed=21):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    one = 0.0 if kind == "gemma" else 1.0
    s = {"X": (randn(T, H) * torch.exp(randn(H))).to(x_type), "F": (randn(T, H) * 3).to(f_type),
         "pre_w": one + 0.2 * randn(H), "post_w": one + 0.2 * randn(H),
         "dX": randn(T, H).to(x_type), "dN": randn(T, H).to(f_type),
         "gate": {"none": None, "token": randn(T, 1), "channel": randn(H)}[gate]}
    return s


def _weight(w, kind):
    return w.double() + 1 if kind == "gemma" else w.double()


def _close(got, ref, err):
    err = 1.01 * err
    bound = err + torch.finfo(got.dtype).eps / 2 * (ref.abs() + err) + 1e-37
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - ref).abs() / bound).max()))


def _check_forward(got, s, kind, alpha, eps):
    X, F = s["X"].double(), s.get("F")
    d = torch.zeros_like(X)
    new = X
    if F is not None:
        P = F.double()
        if s["post_w"] is not None:
            P = P / torch.sqrt((P * P).mean(-1, keepdim=True) + eps) * _weight(s["post_w"], kind)
        P = P if s["gate"] is None else P * s["gate"].double()
        new = alpha * X + P
        d = P.abs() * (R + 6 * U) + 2 * U * ((alpha * X).abs() + P.abs())
        _close(got[0], new, d)
    if s["pre_w"] is None:
        assert got[1] is None
        return
    rx = 1 / torch.sqrt((new * new).mean(-1, keepdim=True) + eps)
    w = _weight(s["pre_w"], kind)
    whole = d.norm(dim=-1, keepdim=True) / new.norm(dim=-1, keepdim=True).clamp(min=1e-300)
    _close(got[1], new * rx * w, (rx * w).abs() * (d + new.abs() * (R + 6 * U + whole)))


def _check_backward(got, s, kind, alpha, eps):
    dX, dF, dpre, dpost, dgate = got
    X = s["X"].double()
    T = 0 * X if s["dX"] is None else s["dX"].double()
    dT = 0 * X
    rows = X.shape[0] + 40
    if s["pre_w"] is not None:
        w, dN = _weight(s["pre_w"], kind), s["dN"].double()
        rx = 1 / torch.sqrt((X * X).mean(-1, keepdim=True) + eps)
        xh, back = X * rx, dN * w
        m = (back * xh).mean(-1, keepdim=True)
        dm = 48 * U * (back * xh).abs().mean(-1, keepdim=True) + m.abs() * (R + 6 * U)
        terms = back.abs() + (xh * m).abs()
        dT = rx * (xh.abs() * dm + terms * (R + 8 * U)) + 4 * U * (T.abs() + rx * terms)
        T = T + rx * (back - xh * m)
        _close(dpre, (dN * xh).sum(0), (dN * xh).abs().sum(0) * (R + 2 * U + rows * U))
    if s.get("F") is None:
        _close(dX, T, dT)
        return
    _close(dX, alpha * T, abs(alpha) * dT + U * (alpha * T).abs())
    F, g = s["F"].double(), 1.0 if s["gate"] is None else s["gate"].double()
    g = torch.as_tensor(g, dtype=torch.float64, device="cuda")
    if s["post_w"] is None:
        rf, fh, w = torch.ones_like(F[:, :1]), F, torch.ones_like(F[0])
    else:
        rf = 1 / torch.sqrt((F * F).mean(-1, keepdim=True) + eps)
        fh, w = F * rf, _weight(s["post_w"], kind)
    if s["gate"] is not None:
        one, each = T * fh * w, dT * (fh * w).abs() + (T * fh * w).abs() * (R + 4 * U)
        if s["gate"].dim() == 2:
            _close(dgate, one.sum(-1, keepdim=True), each.sum(-1, keepdim=True) + 48 * U * one.abs().sum(-1, keepdim=True))
        else:
            _close(dgate, one.sum(0), each.sum(0) + rows * U * one.abs().sum(0))
    if s["post_w"] is None:
        _close(dF, T * g, dT * g.abs() + 2 * U * (T * g).abs())
        return
    one = T * g * fh
    _close(dpost, one.sum(0), (dT * (g * fh).abs() + one.abs() * (R + 4 * U)).sum(0) + rows * U * one.abs().sum(0))
    mf = (one * w).mean(-1, keepdim=True)
    dmf = (dT * (g * w * fh).abs() + (one * w).abs() * (R + 54 * U)).mean(-1, keepdim=True)
    _close(dF, rf * (T * g * w - fh * mf), rf * (dT * (g * w).abs() + fh.abs() * dmf + ((T * g * w).abs() + (fh * mf).abs()) * (R + 8 * U)))


def _both(s, kind="rms", alpha=1.0, eps=1e-5, check=True):
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"], residual_scale=alpha, eps=eps, kind=kind)
    got = capi.sandwich_norm(s["X"], s["F"], **how)
    back = capi.sandwich_norm_backward(s["dX"], s["dN"], s["X"], s["F"], **how)
    if check:
        _check_forward(got, s, kind, alpha, eps)
        _check_backward(back, s, kind, alpha, eps)
    return got, back


@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (7, 200), (1, 2048), (153, 256), (310, 264), (259, 1024), (1000, 1408),
                                 (611, 4096), (5, 4104), (300, 6144), (154, 8192)])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("x_type,f_type", list(itertools.product([BF, F32], [BF, F32])))
def test_both_norms(T, H, gate, x_type, f_type):
    kind, alpha = ("gemma", 0.75) if H % 16 else ("rms", 1.0)
    _both(_inputs(T, H, x_type, f_type, gate, kind), kind, alpha)


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("without", [("pre_w", "dN"), ("post_w",), ("pre_w", "dN", "post_w"), ("dX",)])
@pytest.mark.parametrize("T,H", [(2, 136), (457, 2048), (40, 5000)])
def test_parts(T, H, gate, without):
    s = _inputs(T, H, F32, BF, gate, "rms")
    for name in without:
        s[name] = None
    (new, N), back = _both(s, alpha=-0.5)
    assert (N is None) == (s["pre_w"] is None) and (back[2] is None) == (s["pre_w"] is None)
    assert (back[3] is None) == (s["post_w"] is None) and (back[4] is None) == (s["gate"] is None)


@pytest.mark.parametrize("with_stream", [True, False])
@pytest.mark.parametrize("x_type,n_type", [(F32, BF), (BF, BF), (BF, F32)])
def test_norm_before_the_first_block(x_type, n_type, with_stream):
    s = _inputs(321, 1032, x_type, n_type, "none", "gemma")
    s["F"] = s["post_w"] = None
    if not with_stream:
        s["dX"] = None
    got = capi.sandwich_norm(s["X"], pre_w=s["pre_w"], kind="gemma", n_dtype=n_type)
    assert got[0] is s["X"] and got[1].dtype == n_type
    _check_forward(got, s, "gemma", 1.0, 1e-5)
    back = capi.sandwich_norm_backward(s["dX"], s["dN"], s["X"], pre_w=s["pre_w"], kind="gemma", residual_scale=0.5)
    _check_backward(back, s, "gemma", 1.0, 1e-5)
    assert back[1] is None and back[3] is None and back[4] is None


@pytest.mark.parametrize("factor", [1e37, 1e30, 1e-25, 1e18])
def test_magnitudes(factor):
    """Squares beyond fp32 and below it; the gradients of F fall with 1 / |F|."""
    s = _inputs(64, 520, F32, F32, "channel", "rms")
    s["F"] = s["F"] * factor
    _both(s)
    s["X"] = s["X"] * min(factor, 1e34)  # its largest values are 200 times the others
    s["dX"] = s["dX"] / max(factor, 1.0)
    _both(s, eps=1e-30 if factor < 1 else 1e-5)


def test_zero_rows_and_rows_without_a_norm():
    s = _inputs(9, 264, BF, BF, "none", "rms")
    s["X"][2], s["F"][2], s["F"][5] = 0, 0, 0
    _both(s)
    clean_new, clean_n = _both(s, check=False)[0]
    clean = _both(s, check=False)[1]
    s["F"][4, 7], s["X"][6, 3] = float("nan"), float("inf")
    (new, N), back = _both(s, check=False)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(new[keep], clean_new[keep]) and torch.equal(N[keep], clean_n[keep])
    assert torch.equal(back[0][keep], clean[0][keep]) and torch.equal(back[1][keep], clean[1][keep])
    assert bool(torch.isnan(N[4]).all()) and bool(torch.isnan(back[1][4]).all())
    # inf / inf in its column, finite / inf elsewhere
    assert bool(torch.isnan(N[6, 3])) and bool((N[6, :3] == 0).all())
    assert bool(torch.isnan(back[3]).all())  # the sums over rows hold the row of NaN


def test_gradients_against_differences():
    """Central differences of the fp64 norms along each gradient: their slope is its norm.  Steps of
    2^-12 of the tensor's norm are off by 2^-24 of third derivatives; fp32 results by far less than 2^-12."""
    s = _inputs(23, 136, F32, F32, "token", "gemma")
    eps, alpha = 1e-5, 0.75

    def norm(V, w):
        return V / torch.sqrt((V * V).mean(-1, keepdim=True) + eps) * (1 + w)

    at = {k: s[k].double() for k in ("X", "F", "pre_w", "post_w", "gate")}

    def loss(p):
        new = alpha * p["X"] + p["gate"] * norm(p["F"], p["post_w"])
        return (s["dX"].double() * new).sum() + (s["dN"].double() * norm(new, p["pre_w"])).sum()

    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"], residual_scale=alpha, eps=eps, kind="gemma")
    new, _ = capi.sandwich_norm(s["X"], s["F"], **how)
    grads = dict(zip(("X", "F", "pre_w", "post_w", "gate"), capi.sandwich_norm_backward(s["dX"], s["dN"], new, s["F"], **how)))
    for name, grad in grads.items():
        size = float(grad.double().norm())
        step = 2.0 ** -12 * float(at[name].norm())
        ends = [float(loss({**at, name: at[name] + sign * step * grad.double() / size})) for sign in (1, -1)]
        assert abs((ends[0] - ends[1]) / (2 * step) - size) <= 2.0 ** -10 * size, name


@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (F32, F32)])
def test_in_place_and_again(types):
    s = _inputs(777, 2048, *types, "token", "rms")
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"])
    want = capi.sandwich_norm(s["X"], s["F"], **how)
    back = capi.sandwich_norm_backward(s["dX"], s["dN"], want[0], s["F"], **how)
    again = capi.sandwich_norm_backward(s["dX"], s["dN"], want[0], s["F"], **how)
    assert all(torch.equal(a, b) for a, b in zip(back, again))
    X, F, dX, dN = (s[k].clone() for k in ("X", "F", "dX", "dN"))
    got = capi.sandwich_norm(X, F, X_out=X, N_out=F, **how)
    assert got[0] is X and got[1] is F and torch.equal(X, want[0]) and torch.equal(F, want[1])
    got = capi.sandwich_norm_backward(dX, dN, want[0], s["F"], dX_out=dX, dF_out=dN, **how)
    assert got[0] is dX and got[1] is dN and all(torch.equal(a, b) for a, b in zip(got, back))


def test_no_rows():
    s = _inputs(0, 64, BF, BF, "token", "rms")
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"])
    new, N = capi.sandwich_norm(s["X"], s["F"], **how)
    assert new.shape == N.shape == (0, 64)
    back = capi.sandwich_norm_backward(s["dX"], s["dN"], s["X"], s["F"], **how)
    assert bool((back[2] == 0).all()) and bool((back[3] == 0).all()) and back[4].shape == (0, 1)


def test_captured_and_on_another_stream():
    s = _inputs(300, 1024, F32, BF, "channel", "rms")
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"], residual_scale=0.5)

    def step(stream=None):
        new, N = capi.sandwich_norm(s["X"], s["F"], stream=stream, **how)
        return (new, N) + capi.sandwich_norm_backward(s["dX"], s["dN"], new, s["F"], stream=stream, **how)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    s["X"].mul_(0.5)
    s["dN"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_python_refusals():
    s = _inputs(16, 64, BF, BF, "channel", "rms")
    X, F, w = s["X"], s["F"], s["pre_w"]
    for args, kw in (((X, F[:8]), {}), ((X.half(), F), {}), ((X, F), dict(pre_w=w.double())), ((X, F), dict(pre_w=w[:8])),
                     ((X, F), dict(gate=w.view(1, 64))), ((X, F), dict(kind="layer")), ((X[:, ::2], None), dict(pre_w=w[:32].clone())),
                     ((X, F), dict(N_out=X)), ((X, None), dict(pre_w=w, X_out=F)), ((X.cpu(), F), {}),
                     ((X, F), dict(pre_w=w, n_dtype=F32))):
        with pytest.raises(ValueError):
            capi.sandwich_norm(*args, **kw)
    for kw in (dict(X_out=F), dict(pre_w=w, N_out=X), dict(eps=0.0), dict(residual_scale=float("nan"))):
        with pytest.raises(capi.MoeError):
            capi.sandwich_norm(X, F, **kw)
    with pytest.raises(capi.MoeError):
        capi.sandwich_norm(X)  # nothing to do
    for dX, dN, kw in ((s["dX"], None, dict(pre_w=w)), (s["dX"], s["dN"], {}), (None, None, {}), (s["dX"].float(), None, {})):
        with pytest.raises(ValueError):
            capi.sandwich_norm_backward(dX, dN, X, F, **kw)
    with pytest.raises(capi.MoeError):
        capi.sandwich_norm_backward(s["dX"], None, X, F, dX_out=F, dF_out=X)
