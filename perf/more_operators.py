"""The operators that train an expert layer, as cases to measure.

  grouped_gated_forward / grouped_gated_backward / grouped_gated_dgrad
      H = act(X Wg^T, X Wu^T) over expert-sorted rows (both projections, the activation and
      the product), the gradients of both projections' results from the gradient dY of the
      down projection's result, and the gradient of X from those two
  sandwich_norm / sandwich_norm_backward
      X' = residual_scale X + gate * norm(F) post_w and N = norm(X') pre_w: the norm after a
      block with its gate and the residual, and the norm before the next block; all gradients
  orthogonalize
      Newton-Schulz products that move the singular values of stacked weight gradients
      towards one (the update of the Muon optimiser)

`run` computes each in its plain form, or (`own`) calls the framework.
"""

import math

import torch

own = False  # set from outside: True runs the framework's own operators

DEVICE = "cuda"
TORCH_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ALPHA, LIMIT, BETA = 1.702, 7.0, 1.0  # of the clamped activation
EPS = 1e-5  # of the norms
QUINTIC = (3.4445, -4.7750, 2.0315)  # X <- aX + (bA + cA^2)X, A = XX^T
TINY = 1e-7  # added to the Frobenius norm


# ------------------------------------------------------------------------ cases

def _gated(name, op, T, k, E, I, K, skew, act, out="bf16", save=False, spare=0):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "I": I, "K": K, "skew": skew, "act": act, "out": out,
            "save": save, "spare": spare}


def _norm(name, op, T, H, stream, block, gate, kind, alpha):
    return {"name": name, "op": op, "T": T, "H": H, "stream": stream, "block": block, "gate": gate, "kind": kind,
            "residual_scale": alpha}


def listed():
    return [
        # one decoded token: the gate and up projections of six experts are streamed once
        _gated("gated forward one token", "forward", 1, 6, 64, 1408, 2048, False, "silu"),
        # a training or prefill batch, both projections kept for the backward pass
        _gated("gated forward batch", "forward", 4096, 6, 64, 1408, 2048, False, "silu", save=True),
        # a small layer whose sizes divide by nothing, some experts unused, clamped activation
        _gated("gated backward small odd", "backward", 259, 3, 16, 200, 328, True, "swigluoai", spare=23),
        # the backward pass of a training batch through the down projection and the activation
        _gated("gated backward batch", "backward", 4096, 6, 64, 1408, 2048, False, "silu"),
        # input gradient of many small experts at a short batch
        _gated("gated dgrad small experts", "dgrad", 250, 8, 128, 256, 1024, True, "silu"),
        # input gradient of a training batch, tokens crowding on a few experts, summed on in fp32
        _gated("gated dgrad skewed batch", "dgrad", 4096, 6, 64, 1408, 2048, True, "silu", out="f32"),
        # between two blocks while decoding one token
        _norm("norms one token", "norm", 1, 2048, "bf16", "bf16", "none", "rms", 1.0),
        # between two blocks of a prefill batch whose residual stream is kept in fp32, tokens gated
        _norm("norms batch", "norm", 8192, 2048, "f32", "bf16", "token", "rms", 1.0),
        # all gradients between two blocks of a short batch, a gate for each channel
        _norm("norms backward short", "norm_backward", 251, 1024, "bf16", "bf16", "channel", "gemma", 0.75),
        # all gradients between two blocks of a training batch
        _norm("norms backward batch", "norm_backward", 16384, 2048, "bf16", "bf16", "none", "rms", 1.0),
        # the update of one small projection
        {"name": "orthogonalise one matrix", "op": "orthogonalize", "E": 1, "N": 256, "K": 1024, "steps": 5, "type": "f32"},
        # the update of half a layer's stacked experts
        {"name": "orthogonalise experts", "op": "orthogonalize", "E": 32, "N": 1408, "K": 2048, "steps": 5, "type": "f32"},
    ]


def _log_int(rng, low, high, step=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step))


def draw(rng):
    op = rng.choice(["forward", "backward", "dgrad", "norm", "norm_backward", "orthogonalize"])
    largest = [work(c) for c in listed() if c["op"] == op]
    flops, size = max(w["flops"] for w in largest), max(w["bytes"] for w in largest)
    while True:
        if op == "orthogonalize":
            case = {"op": op, "E": _log_int(rng, 1, 64), "N": _log_int(rng, 64, 4096, 8), "K": _log_int(rng, 64, 4096, 8),
                    "steps": rng.choice([5, 5, 4, 6]), "type": rng.choice(["bf16", "f32"])}
        elif op in ("norm", "norm_backward"):
            case = {"op": op, "T": _log_int(rng, 1, 60000), "H": _log_int(rng, 64, 8192, 8),
                    "stream": rng.choice(["bf16", "f32"]), "block": rng.choice(["bf16", "bf16", "f32"]),
                    "gate": rng.choice(["none", "token", "channel"]), "kind": rng.choice(["rms", "gemma"]),
                    "residual_scale": rng.choice([1.0, 1.0, 0.75])}
        else:
            E = _log_int(rng, 1, 128)
            case = {"op": op, "T": _log_int(rng, 1, 8192), "k": rng.randint(1, min(E, 8)), "E": E,
                    "I": _log_int(rng, 64, 4096, 8), "K": _log_int(rng, 64, 4096, 8), "skew": rng.random() < 0.5,
                    "act": rng.choice(["silu", "swigluoai"]), "out": rng.choice(["bf16", "f32"]) if op == "dgrad" else "bf16",
                    "save": op == "forward" and rng.random() < 0.5, "spare": rng.choice([0, 0, rng.randint(1, 300)])}
        w = work(case)
        if w["flops"] <= flops and w["bytes"] <= size and w["bytes"] > 2e4:
            return case


def work(case):
    op = case["op"]
    if op == "orthogonalize":
        E, m, n = case["E"], min(case["N"], case["K"]), max(case["N"], case["K"])
        # XX^T and its square are symmetric: half of their products; the product with X is whole
        step = m * m * n + m * m * m + 2 * m * m * n
        return {"bytes": E * m * n * (2 + (2 if case["type"] == "bf16" else 4)), "flops": E * case["steps"] * step}
    if op in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]
        x, f = (2 if case[t] == "bf16" else 4 for t in ("stream", "block"))
        gate = {"none": 0, "token": 4 * T, "channel": 4 * H}[case["gate"]]
        if op == "norm":  # X and F in, X' and N out
            return {"bytes": T * H * (2 * x + 2 * f) + 8 * H + gate, "flops": 12 * T * H}
        # X', F, dX' and dN in, dX and dF out, and the gradients of the weights and the gate
        return {"bytes": T * H * (3 * x + 3 * f) + 2 * (8 * H + gate), "flops": 30 * T * H}
    R, E, I, K = case["T"] * case["k"], case["E"], case["I"], case["K"]
    touched = E * (1 - (1 - case["k"] / E) ** case["T"])  # experts that receive a row
    out = 2 if case["out"] == "bf16" else 4
    b = {"forward": R * K * 2 + touched * 2 * I * K * 2 + R * I * 2 * (3 if case["save"] else 1),
         "backward": R * K * 2 + touched * I * K * 2 + R * I * 2 * 4,
         "dgrad": R * I * 2 * 2 + touched * 2 * I * K * 2 + R * K * out}[op]
    return {"bytes": b, "flops": 2 * R * I * K * (1 if op == "backward" else 2)}


# ----------------------------------------------------------------------- inputs

def _routing(case, gen):
    """Row counts of the experts when every token takes its k best of noisy scores."""
    T, k, E = case["T"], case["k"], case["E"]
    scores = torch.sigmoid(torch.randn(T, E, generator=gen, device=DEVICE))
    if case["skew"]:  # a few experts are preferred: r^-1.2 over a random order of the experts
        bias = torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32) ** -1.2
        scores += 0.5 * bias[torch.randperm(E, generator=gen, device=DEVICE)]
    return torch.bincount(scores.topk(k, dim=1).indices.flatten(), minlength=E)


def _normal(gen, shape, std, dtype):
    out = torch.empty(shape, dtype=dtype, device=DEVICE)
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 26) // flat.shape[1])
    for i in range(0, flat.shape[0], step):  # bounds the fp32 temporary
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEVICE) * std)
    return out


def _stream(gen, T, H, dtype):
    """Hidden states: a few channels are far larger than the others."""
    channel = torch.exp(0.3 * torch.randn(H, generator=gen, device=DEVICE))
    channel[torch.randperm(H, generator=gen, device=DEVICE)[:max(1, H // 256)]] *= 20
    return _normal(gen, (T, H), channel, dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "orthogonalize":
        # directions of falling weight under noise, as a momentum of gradients has them
        E, N, K = case["E"], case["N"], case["K"]
        G = torch.empty(E, N, K, dtype=TORCH_TYPE[case["type"]], device=DEVICE)
        r = min(N, K)
        weight = torch.arange(1, r + 1, device=DEVICE, dtype=torch.float32) ** -0.5
        for e in range(E):
            left = torch.randn(N, r, generator=gen, device=DEVICE) * weight
            right = torch.randn(r, K, generator=gen, device=DEVICE)
            G[e] = 1e-3 * (left @ right + torch.randn(N, K, generator=gen, device=DEVICE))
        s["G"], s["steps"] = G, case["steps"]
        s["out"] = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEVICE)
        return s
    if op in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]
        stream, block = TORCH_TYPE[case["stream"]], TORCH_TYPE[case["block"]]
        one = 0.0 if case["kind"] == "gemma" else 1.0
        s.update(kind=case["kind"], residual_scale=case["residual_scale"], gate=None)
        s["X"], s["F"] = _stream(gen, T, H, stream), _stream(gen, T, H, block)
        s["pre_w"] = one + 0.1 * torch.randn(H, generator=gen, device=DEVICE)
        s["post_w"] = one + 0.1 * torch.randn(H, generator=gen, device=DEVICE)
        if case["gate"] != "none":
            n = T if case["gate"] == "token" else H
            s["gate"] = torch.sigmoid(torch.randn(n, generator=gen, device=DEVICE))
            s["gate"] = s["gate"].view(T, 1) if case["gate"] == "token" else s["gate"]
        if op == "norm_backward":
            s["dX"], s["dN"] = _normal(gen, (T, H), 0.01, stream), _normal(gen, (T, H), 0.01, block)
        return s
    E, I, K = case["E"], case["I"], case["K"]
    counts = _routing(case, gen)
    s["offs"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["max_rows"] = int(counts.max())
    s["act"], s["type"], s["save"] = case["act"], TORCH_TYPE[case["out"]], case["save"]
    rows = case["T"] * case["k"] + case["spare"]  # the buffers hold `spare` rows that no expert owns
    if op == "forward":
        s["X"] = _normal(gen, (rows, K), 1.0, torch.bfloat16)
    if op != "backward":
        s["Wg"], s["Wu"] = (_normal(gen, (E, I, K), 0.02, torch.bfloat16) for _ in range(2))
    if op == "backward":
        s["dY"] = _normal(gen, (rows, K), 0.01, torch.bfloat16)
        s["Wd"] = _normal(gen, (E, K, I), 0.02, torch.bfloat16)
        # what products over K give; the clamped activation's limit is passed now and then
        s["G"], s["U"] = (_normal(gen, (rows, I), 3.0 if case["act"] == "swigluoai" else 1.0, torch.bfloat16) for _ in range(2))
    if op == "dgrad":
        s["dG"], s["dU"] = (_normal(gen, (rows, I), 0.01, torch.bfloat16) for _ in range(2))
        s["outs"] = [torch.zeros(rows, K, dtype=s["type"], device=DEVICE)]
    else:
        n = 2 if op == "backward" else 3 if s["save"] else 1
        s["outs"] = [torch.zeros(rows, I, dtype=torch.bfloat16, device=DEVICE) for _ in range(n)]
    return s


# ------------------------------------------------------------------ plain forms

def _padded(s, rows):
    """[E, max_rows] row numbers of each expert, those it does not own pointing past the rows."""
    at = s["offs"][:-1, None].long() + torch.arange(max(1, s["max_rows"]), device=DEVICE)
    return torch.where(at < s["offs"][1:, None], at, rows)


def _by_expert(A, at):
    return torch.cat([A.float(), A.new_zeros(1, A.shape[1], dtype=torch.float32)])[at]


def _store(out, at, got):
    """The experts' rows of out; the others stay as they are."""
    whole = torch.cat([out, out.new_zeros(1, out.shape[1])])
    whole[at] = got.to(out.dtype)
    out.copy_(whole[:-1])


def _plain_gated(s):
    op = s["op"]
    if op == "forward":
        at = _padded(s, s["X"].shape[0])
        X = _by_expert(s["X"], at)
        g, u = (torch.bmm(X, s[w].float().transpose(1, 2)) for w in ("Wg", "Wu"))
        if s["act"] == "silu":
            h = g / (1 + torch.exp(-g)) * u
        else:
            gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
            h = gc / (1 + torch.exp(-ALPHA * gc)) * (uc + BETA)
        results = (h, g, u)
    elif op == "backward":
        at = _padded(s, s["dY"].shape[0])
        dh = torch.bmm(_by_expert(s["dY"], at), s["Wd"].float())
        g, u = _by_expert(s["G"], at), _by_expert(s["U"], at)
        if s["act"] == "silu":
            sig = 1 / (1 + torch.exp(-g))
            results = (dh * u * (sig * (1 + g * (1 - sig))), dh * (g * sig))
        else:
            gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
            sig = 1 / (1 + torch.exp(-ALPHA * gc))
            dg = dh * (uc + BETA) * (sig * (1 + ALPHA * gc * (1 - sig)))
            results = (torch.where(g <= LIMIT, dg, 0.0), torch.where(u.abs() <= LIMIT, dh * (gc * sig), 0.0))
    else:
        at = _padded(s, s["dG"].shape[0])
        results = (torch.bmm(_by_expert(s["dG"], at), s["Wg"].float()) + torch.bmm(_by_expert(s["dU"], at), s["Wu"].float()),)
    for out, got in zip(s["outs"], results):
        _store(out, at, got)
    return s["outs"]


def _effective(w, s):
    return w + 1 if s["kind"] == "gemma" else w


def _plain_norm(s):
    X, F = s["X"].float(), s["F"].float()
    pre, post = _effective(s["pre_w"], s), _effective(s["post_w"], s)
    gate = 1.0 if s["gate"] is None else s["gate"]
    rf = torch.rsqrt(F.square().mean(-1, keepdim=True) + EPS)
    if s["op"] == "norm":
        new = s["residual_scale"] * X + gate * (F * rf * post)
        N = new * torch.rsqrt(new.square().mean(-1, keepdim=True) + EPS) * pre
        return new.to(s["X"].dtype), N.to(s["F"].dtype)
    dN = s["dN"].float()
    rx = torch.rsqrt(X.square().mean(-1, keepdim=True) + EPS)
    xhat, back = X * rx, dN * pre
    total = s["dX"].float() + rx * (back - xhat * (back * xhat).mean(-1, keepdim=True))
    fhat = F * rf
    dP = total * gate
    back = dP * post
    dF = rf * (back - fhat * (back * fhat).mean(-1, keepdim=True))
    dgate = None
    if s["gate"] is not None:
        of = total * (fhat * post)
        dgate = of.sum(-1, keepdim=True) if s["gate"].dim() == 2 else of.double().sum(0).float()
    return ((s["residual_scale"] * total).to(s["X"].dtype), dF.to(s["F"].dtype), (dN * xhat).double().sum(0).float(),
            (dP * fhat).double().sum(0).float(), dgate)


def _plain_orthogonalize(s):
    a, b, c = QUINTIC
    X = s["G"].float()
    tall = X.shape[1] > X.shape[2]
    X = X / (X.double().square().sum((1, 2), keepdim=True).sqrt() + TINY).float()
    if tall:
        X = X.transpose(1, 2)
    for _ in range(s["steps"]):
        A = torch.bmm(X, X.transpose(1, 2))
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    s["out"].copy_(X.transpose(1, 2) if tall else X)
    return s["out"]


# ------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        plain = {"norm": _plain_norm, "norm_backward": _plain_norm, "orthogonalize": _plain_orthogonalize}
        return plain.get(op, _plain_gated)(s)
    from expert_routed_ffn_gb300 import capi
    if op == "forward":
        H, *saved = s["outs"]
        capi.grouped_gated_forward(s["X"], s["Wg"], s["Wu"], s["offs"], act=s["act"], out=H,
                                   save=tuple(saved) if s["save"] else None)
        return s["outs"]
    if op == "backward":
        capi.grouped_gated_backward(s["dY"], s["Wd"], s["G"], s["U"], s["offs"], act=s["act"], out=tuple(s["outs"]))
        return s["outs"]
    if op == "dgrad":
        capi.grouped_gated_dgrad(s["dG"], s["dU"], s["Wg"], s["Wu"], s["offs"], out=s["outs"][0])
        return s["outs"]
    if op == "orthogonalize":
        return capi.orthogonalize(s["G"], steps=s["steps"], coefficients=QUINTIC, eps=TINY, out=s["out"])
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"], residual_scale=s["residual_scale"], eps=EPS, kind=s["kind"])
    if op == "norm":
        return capi.sandwich_norm(s["X"], s["F"], **how)
    return capi.sandwich_norm_backward(s["dX"], s["dN"], s["X"], s["F"], **how)


# ------------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "orthogonalize":
        a, b, c = QUINTIC
        out = torch.empty(s["G"].shape, dtype=torch.float64, device=DEVICE)
        for e, G in enumerate(s["G"]):
            X = G.double()
            X = X / (torch.sqrt((X * X).sum()) + TINY)
            for _ in range(s["steps"]):  # from the smaller side: the same polynomial of the singular values
                if X.shape[0] <= X.shape[1]:
                    A = X @ X.t()
                    X = a * X + b * (A @ X) + c * (A @ (A @ X))
                else:
                    A = X.t() @ X
                    X = a * X + b * (X @ A) + c * ((X @ A) @ A)
            out[e] = X
        return out
    if op in ("norm", "norm_backward"):
        return _exact_norm(s)
    offs = s["offs"].tolist()
    outs = [torch.zeros(o.shape, dtype=torch.float64, device=DEVICE) for o in s["outs"]]
    for e in range(case["E"]):
        r = slice(offs[e], offs[e + 1])
        if op == "forward":
            g, u = s["X"][r].double() @ s["Wg"][e].double().t(), s["X"][r].double() @ s["Wu"][e].double().t()
            got = (_exact_act(g, u, s["act"]), g, u)
        elif op == "backward":
            g, u = (s[n][r].double().requires_grad_() for n in ("G", "U"))
            dh = s["dY"][r].double() @ s["Wd"][e].double()
            got = torch.autograd.grad(_exact_act(g, u, s["act"]), (g, u), dh)
        else:
            got = (s["dG"][r].double() @ s["Wg"][e].double() + s["dU"][r].double() @ s["Wu"][e].double(),)
        for o, v in zip(outs, got):
            o[r] = v
    return outs


def _exact_act(g, u, act):
    if act == "silu":
        return g * torch.sigmoid(g) * u
    g, u = torch.clamp(g, max=LIMIT), torch.clamp(u, min=-LIMIT, max=LIMIT)
    return g * torch.sigmoid(ALPHA * g) * (u + BETA)


def _exact_norm(s):
    """The definition, its gradients by automatic differentiation."""
    def norm(V, w):
        return V / torch.sqrt((V * V).mean(-1, keepdim=True) + EPS) * (w + 1 if s["kind"] == "gemma" else w)

    pre, post = s["pre_w"].double().requires_grad_(), s["post_w"].double().requires_grad_()
    gate = None if s["gate"] is None else s["gate"].double().requires_grad_()
    F, X = s["F"].double().requires_grad_(), s["X"].double()
    branch = norm(F, post) if gate is None else gate * norm(F, post)
    if s["op"] == "norm":
        new = s["residual_scale"] * X + branch
        return new.detach(), norm(new, pre).detach()
    # X is what the block gave, X = residual_scale X_in + branch
    X.requires_grad_()
    to_stream, dpre = torch.autograd.grad(norm(X, pre), (X, pre), s["dN"].double())
    total = s["dX"].double() + to_stream
    wanted = [F, post] + ([] if gate is None else [gate])
    dF, dpost, *dgate = torch.autograd.grad(branch, wanted, total)
    return s["residual_scale"] * total, dF, dpre, dpost, (dgate[0] if dgate else None)
