"""A training step of an expert layer, made of the operators as a program would call them: the norm
before, the experts' gated projections and the down projection on the dispatch's rows, the norm
after with gate and residual, all gradients back, clipping, and the orthogonalised update.

Against fp64 autograd of the same step.  A tensor between two operators is rounded to bf16 once: off
by at most 2^-9 of its values, which later steps pass on as they pass on the values themselves; the
longest path (norm, G and U, H, Y, F, N, their gradients dF, dY, dG, dU, dX and the sums over
tokens) has 14 such roundings, so 14 * 2^-9 of a gradient's 2-norm.
"""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, H, E, K, I = 203, 264, 7, 2, 136
ROUNDINGS = 14 * 2.0 ** -9


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


def _setup(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    p = {"pre": 1 + randn(H, std=0.1), "post": 1 + randn(H, std=0.1), "next": 1 + randn(H, std=0.1), "gate": randn(H),
         "Wg": randn(E, I, H, std=0.08).to(BF), "Wu": randn(E, I, H, std=0.08).to(BF), "Wd": randn(E, H, I, std=0.08).to(BF)}
    X = randn(T, H)
    # every token takes K of the experts but the last, which none takes
    experts = torch.rand(T, E - 1, generator=gen, device="cuda").topk(K, dim=1).indices
    weight = torch.rand(T, K, generator=gen, device="cuda") + 0.1
    order = experts.flatten().argsort(stable=True)
    counts = torch.bincount(experts.flatten(), minlength=E)
    route = {"token": order // K, "weight": weight.flatten()[order].unsqueeze(1), "order": order,
             "offs": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)}
    return p, X, route, randn(T, H), randn(T, H).to(BF)


def _step(p, X, route, dXn, dN, act):
    """(X', N, gradients by name) by the operators."""
    token, weight, offs = route["token"], route["weight"], route["offs"]
    _, N0 = capi.sandwich_norm(X, pre_w=p["pre"], n_dtype=BF)
    rows = N0[token]
    Hid, G, U = capi.grouped_gated_forward(rows, p["Wg"], p["Wu"], offs, act=act, save=True)
    Y = capi.grouped_forward(Hid, p["Wd"], offs)
    F = torch.zeros(T, H, device="cuda").index_add_(0, token, weight * Y.float()).to(BF)
    how = dict(pre_w=p["next"], post_w=p["post"], gate=p["gate"], residual_scale=0.75)
    Xn, N = capi.sandwich_norm(X, F, **how)

    dX, dF, dnext, dpost, dgate = capi.sandwich_norm_backward(dXn, dN, Xn, F, **how)
    dY = (weight * dF[token].float()).to(BF)
    dG, dU = capi.grouped_gated_backward(dY, p["Wd"], G, U, offs, act=act)
    drows = capi.grouped_gated_dgrad(dG, dU, p["Wg"], p["Wu"], offs, out_dtype=torch.float32)
    dN0 = torch.zeros(T, H, device="cuda").index_add_(0, token, drows).to(BF)
    dX, _, dpre, _, _ = capi.sandwich_norm_backward(dX, dN0, X, pre_w=p["pre"])
    return Xn, N, {"X": dX, "pre": dpre, "post": dpost, "next": dnext, "gate": dgate, "Wg": capi.grouped_wgrad(dG, rows, offs),
                   "Wu": capi.grouped_wgrad(dU, rows, offs), "Wd": capi.grouped_wgrad(dY, Hid, offs)}


def _reference(p, X, route, dXn, dN, act):
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    x = X.double().requires_grad_()

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w

    token, o = route["token"], route["offs"].tolist()
    rows = norm(x, q["pre"])[token]
    Y = []
    for e in range(E):
        g, u = rows[o[e]:o[e + 1]] @ q["Wg"][e].t(), rows[o[e]:o[e + 1]] @ q["Wu"][e].t()
        if act == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            g, u = g.clamp(max=7.0), u.clamp(-7.0, 7.0)
            h = g * torch.sigmoid(1.702 * g) * (u + 1)
        Y.append(h @ q["Wd"][e].t())
    F = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add(0, token, route["weight"].double() * torch.cat(Y))
    new = 0.75 * x + q["gate"] * norm(F, q["post"])
    N = norm(new, q["next"])
    loss = (dXn.double() * new).sum() + (dN.double() * N).sum()
    names = ["X"] + list(p)
    grads = torch.autograd.grad(loss, [x] + list(q.values()))
    return new.detach(), N.detach(), dict(zip(names, grads))


@pytest.mark.parametrize("act", ["silu", "swigluoai"])
def test_against_autograd(act):
    s = _setup(41)
    Xn, N, got = _step(*s, act)
    want_x, want_n, want = _reference(*s, act)
    for name, a, b in [("X'", Xn, want_x), ("N", N, want_n)] + [(k, got[k], want[k]) for k in want]:
        error, size = float((a.double() - b).norm()), float(b.norm())
        assert error <= ROUNDINGS * size, (name, error / size)
    assert bool((got["Wg"][E - 1] == 0).all())  # the expert that no token took


def _polynomial(G):
    X = G / (G.flatten(1).norm(dim=1)[:, None, None] + 1e-7)
    for _ in range(5):
        A = X @ X.transpose(1, 2)
        X = 3.4445 * X + (-4.7750 * A + 2.0315 * A @ A) @ X
    return X


def test_update_and_next_step():
    """Clipping and the orthogonalised update of the experts' weights, then the step again; the whole
    of it captured and replayed gives the same."""
    p, X, route, dXn, dN = _setup(42)
    start = {k: v.clone() for k, v in p.items()}

    def train():
        _, _, grads = _step(p, X, route, dXn, dN, "silu")
        norm = capi.clip_grad_norm([g for k, g in grads.items() if k != "X"], 1.0)
        updates = []
        for name in ("Wg", "Wu", "Wd"):
            O = capi.orthogonalize(grads[name])
            p[name].sub_(0.02 * O)
            updates.append(O)
        return norm, updates, grads

    norm, updates, grads = train()
    assert float(norm) > 1.0
    for name, O in zip(("Wg", "Wu", "Wd"), updates):
        # an expert's gradient has the rank of its rows, fewer than its sides; the bound is that of
        # tests/test_gpu_orthogonalize.py: 24 roundings to fp16, and one to bf16
        ref = _polynomial(grads[name].double())
        assert float((O.double() - ref).norm()) <= (24 * 2.0 ** -12 + 2.0 ** -8) * float(ref.norm()), name
        assert bool((O[E - 1] == 0).all()) and not torch.equal(p[name][0], start[name][0])
        assert torch.equal(p[name][E - 1], start[name][E - 1])
    after = {k: v.clone() for k, v in p.items()}

    for k in p:
        p[k].copy_(start[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = train()
    for k in p:
        p[k].copy_(start[k])
    graph.replay()
    torch.cuda.synchronize()
    # torch's index_add_ adds in no fixed order: what follows it is the same up to its roundings
    for name, O in zip(("Wg", "Wu", "Wd"), captured[1]):
        assert float((p[name].float() - after[name].float()).norm()) <= ROUNDINGS * float(after[name].float().norm())
    assert abs(float(captured[0]) - float(norm)) <= ROUNDINGS * float(norm)
    train()
    assert all(bool(torch.isfinite(v.float()).all()) for v in p.values())
