"""The operators around the stacked expert weights, as cases to measure.

  grouped_forward / grouped_dgrad / grouped_wgrad
      the products of an MoE layer's expert-sorted rows with the stacked weights
      [E, N, K], and their two gradients; rows of expert e are [offs[e], offs[e + 1])
  mx_quantize -> mx_dequantize
      a tensor to OCP microscaling codes with one power-of-two scale per 32 values, and
      the values those codes stand for (quantisation-aware training and checking)
  mx_quantize -> mx_grouped_forward
      bf16 tokens quantised to MXFP4 and multiplied with MXFP4 expert weights
  clip_grad_norm
      the global norm of a list of gradients and the clipped gradients

`run` computes each in its plain form, or (`own`) calls the framework.
"""

import math

import torch

own = False  # set from outside: True runs the framework's own operators

DEVICE = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
TORCH_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------ cases

def _grouped(name, op, T, k, E, N, K, skew, out, spare=0):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "skew": skew, "out": out, "spare": spare}


def listed():
    return [
        # the gate projection of one decoded token: six experts' weights are streamed once
        _grouped("forward one token", "forward", 1, 6, 64, 1408, 2048, False, "bf16"),
        # the gate projection of a prefill batch
        _grouped("forward prefill", "forward", 4096, 6, 64, 1408, 2048, False, "bf16"),
        # input gradient of a small layer whose sizes divide by nothing, some experts unused
        _grouped("dgrad small odd", "dgrad", 259, 3, 16, 328, 200, True, "f32", 23),
        # input gradient of the down projection, tokens crowding on a few experts
        _grouped("dgrad skewed batch", "dgrad", 4096, 6, 64, 2048, 1408, True, "bf16"),
        # weight gradient of small experts at a short batch: many experts see few rows or none
        _grouped("wgrad small experts", "wgrad", 250, 8, 128, 256, 1024, True, "bf16"),
        # weight gradient of a prefill-sized batch into fp32 main gradients
        _grouped("wgrad batch", "wgrad", 4096, 6, 64, 1408, 2048, False, "f32"),
        # MXFP4 tokens x MXFP4 weights: a decode batch and a prefill batch
        _grouped("mxfp4 decode batch", "mx_forward", 64, 6, 64, 2048, 1408, False, "f32"),
        _grouped("mxfp4 prefill", "mx_forward", 4096, 6, 64, 1408, 2048, False, "bf16"),
        # the tokens of a decode batch, and one projection of all experts (a checkpoint's tensor)
        {"name": "quantise tokens mxfp8", "op": "quantize", "slices": 1, "rows": 251, "K": 1024, "format": "mxfp8", "type": "f32"},
        {"name": "quantise weights mxfp4", "op": "quantize", "slices": 64, "rows": 1408, "K": 2048, "format": "mxfp4", "type": "bf16"},
        # the gradients of a small model's many tensors, and of a large layer's stacked experts
        {"name": "clip many small", "op": "clip", "tensors": 301, "total": 5_000_003, "type": "mixed", "norm_to": 0.5},
        {"name": "clip experts", "op": "clip", "tensors": 5, "total": 553_000_007, "type": "f32", "norm_to": 0.25},
    ]


def _log_int(rng, low, high, step=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step))


def draw(rng):
    op = rng.choice(["forward", "dgrad", "wgrad", "mx_forward", "quantize", "clip"])
    largest = [work(c) for c in listed() if c["op"] == op]
    flops, size = max(w["flops"] for w in largest), max(w["bytes"] for w in largest)
    while True:
        if op == "quantize":
            case = {"op": op, "slices": rng.choice([1, 1, 3, 16, 64]), "rows": _log_int(rng, 1, 20000),
                    "K": _log_int(rng, 32, 6144, 32), "format": rng.choice(["mxfp4", "mxfp4", "mxfp8"]),
                    "type": rng.choice(["bf16", "f32"])}
        elif op == "clip":
            case = {"op": op, "tensors": _log_int(rng, 1, 600), "total": _log_int(rng, 5000, 400_000_000),
                    "type": rng.choice(["bf16", "f32", "mixed"]), "norm_to": rng.choice([0.1, 0.5, 2.0])}
        else:
            E = _log_int(rng, 1, 128)
            step = 32 if op == "mx_forward" else 8
            case = {"op": op, "T": _log_int(rng, 1, 8192), "k": rng.randint(1, min(E, 8)), "E": E,
                    "N": _log_int(rng, 64, 4096, 8), "K": _log_int(rng, 64, 4096, step), "skew": rng.random() < 0.5,
                    "out": rng.choice(["bf16", "f32"]), "spare": rng.choice([0, 0, rng.randint(1, 300)])}
        w = work(case)
        if w["flops"] <= flops and w["bytes"] <= size and w["bytes"] > 1e5:
            return case


def work(case):
    op = case["op"]
    if op == "clip":
        per = {"bf16": 2, "f32": 4, "mixed": 3}[case["type"]]
        return {"bytes": 2 * per * case["total"], "flops": 3 * case["total"]}
    if op == "quantize":
        n = case["slices"] * case["rows"] * case["K"]
        per = 2 if case["type"] == "bf16" else 4
        code = 0.5 if case["format"] == "mxfp4" else 1.0
        # the tensor in, codes and scales out; the values of the codes (the same type) out
        return {"bytes": n * (2 * per + code + 1 / 32), "flops": 4 * n}
    R, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
    touched = E * (1 - (1 - case["k"] / E) ** case["T"])  # experts that receive a row
    out = 2 if case["out"] == "bf16" else 4
    b = {"forward": R * K * 2 + touched * N * K * 2 + R * N * out,
         "dgrad": R * N * 2 + touched * N * K * 2 + R * K * out,
         "wgrad": R * (N + K) * 2 + E * N * K * out,
         "mx_forward": R * K * 2 + touched * N * K * 17 / 32 + R * N * out}[op]
    return {"bytes": b, "flops": 2 * R * N * K}


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
    flat = out.view(-1, shape[-1]) if len(shape) > 1 else out.view(1, -1)
    step = max(1, (1 << 26) // flat.shape[1])
    for i in range(0, flat.shape[0], step):  # bounds the fp32 temporary
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEVICE) * std)
    return out


def _quantize_weights(W):
    """MXFP4 codes [E, N, K / 2] and scales [E, K / 32, N], as a checkpoint stores them."""
    parts = [_mx_plain(W[i:i + 8], "mxfp4") for i in range(0, W.shape[0], 8)]
    codes = torch.cat([_pack(p[0]) for p in parts])
    return codes, torch.cat([p[2] for p in parts])


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "clip":
        n, total = case["tensors"], case["total"]
        # a few large matrices and many vectors, in the order of a model's layers (the same for every seed)
        share = torch.rand(n, generator=torch.Generator().manual_seed(n), dtype=torch.float64) ** 4 + 1e-4
        sizes = (share / share.sum() * (total - n)).long().add_(1).tolist()
        sizes[0] += total - sum(sizes)
        kinds = [("bf16", "f32")[i % 2] if case["type"] == "mixed" else case["type"] for i in range(n)]
        # views of one flat buffer for each type, every view at a multiple of 8 elements
        s["flat"], s["flat_out"], s["grads"], s["out"] = [], [], [], []
        for kind in sorted(set(kinds)):
            starts, end = [], 0
            for m, of in zip(sizes, kinds):
                starts.append(end)
                end += -(-m // 8) * 8 if of == kind else 0
            flat = torch.zeros(end, dtype=TORCH_TYPE[kind], device=DEVICE)
            out = torch.zeros_like(flat)
            for i, (m, of, at) in enumerate(zip(sizes, kinds, starts)):
                if of != kind:
                    continue
                for j in range(0, m, 1 << 27):
                    part = flat[at + j:at + min(m, j + (1 << 27))]
                    part.copy_(torch.randn(part.shape, generator=gen, device=DEVICE) * (1e-3 * (1 + i % 7)))
                s["grads"].append(flat[at:at + m])
                s["out"].append(out[at:at + m])
            s["flat"].append(flat)
            s["flat_out"].append(out)
        parts = torch.stack([torch.linalg.vector_norm(g, dtype=torch.float32) for g in s["grads"]])
        s["max_norm"] = case["norm_to"] * float(parts.norm())  # under 1: clipped; over 1: passed through
        return s
    if op == "quantize":
        s["format"] = case["format"]
        shape = (case["slices"], case["rows"], case["K"])
        s["X"] = _normal(gen, shape, 0.02 if case["slices"] > 1 else 1.0, TORCH_TYPE[case["type"]])
        return s
    E, N, K = case["E"], case["N"], case["K"]
    counts = _routing(case, gen)
    s["offs"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["max_rows"] = int(counts.max())
    s["type"] = TORCH_TYPE[case["out"]]
    rows = case["T"] * case["k"] + case["spare"]  # the buffers hold `spare` rows that no expert owns
    if op != "dgrad":
        s["X"] = _normal(gen, (rows, K), 1.0, torch.bfloat16)
    if op in ("dgrad", "wgrad"):
        s["dY"] = _normal(gen, (rows, N), 0.01, torch.bfloat16)
    if op != "wgrad":
        W = _normal(gen, (E, N, K), 0.02, torch.bfloat16)
        if op == "mx_forward":
            s["Wc"], s["Ws"] = _quantize_weights(W)
        else:
            s["W"] = W
        s["out"] = torch.zeros(rows, K if op == "dgrad" else N, dtype=s["type"], device=DEVICE)
    else:
        s["out"] = torch.zeros(E, N, K, dtype=s["type"], device=DEVICE)
    return s


# ------------------------------------------------------------------ plain forms

def _pack(mag_sign):
    return mag_sign[..., 0::2] | (mag_sign[..., 1::2] << 4)


def _mx_plain(X, fmt):
    """[.., rows, K] -> element codes as whole numbers, their values, scales [.., K / 32, rows]."""
    x = X.float().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1)
    exponent = torch.frexp(amax).exponent - 1 - (2 if fmt == "mxfp4" else 8)
    exponent = torch.where(amax > 0, exponent, -127).clamp(min=-127)
    v = torch.ldexp(x, -exponent.unsqueeze(-1))
    if fmt == "mxfp4":
        a = v.abs().clamp(max=6.0)
        mid = torch.tensor(E2M1_MID, device=X.device)
        low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
        code = torch.where((low & 1) == 0, low, high)  # a value half way goes to the even code
        value = torch.tensor(E2M1, device=X.device)[code].copysign(v)
        code = (code + 8 * torch.signbit(v)).to(torch.uint8)
    else:
        value = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        code, value = value.view(torch.uint8), value.float()
    scale = (exponent + 127).to(torch.uint8).transpose(-1, -2).contiguous()
    return code.flatten(-2), torch.ldexp(value, exponent.unsqueeze(-1)).flatten(-2), scale


def _mx_values(codes, scales):
    """The values of MXFP4 codes [.., rows, K / 2] with scales [.., K / 32, rows], in fp32."""
    table = torch.tensor(E2M1, device=codes.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    e = scales.transpose(-1, -2).float() - 127
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(e).unsqueeze(-1)).flatten(-2)


def _padded(s, rows):
    """[E, max_rows] row numbers of each expert, and which of them it owns."""
    at = s["offs"][:-1, None].long() + torch.arange(max(1, s["max_rows"]), device=DEVICE)
    mine = at < s["offs"][1:, None]
    return torch.where(mine, at, rows), mine


def _by_expert(A, at):
    return torch.cat([A.float(), A.new_zeros(1, A.shape[1], dtype=torch.float32)])[at]


def _products(s, A, W):
    """out[r] = A[r] W[e] for the rows r of expert e; the others stay as they are."""
    rows = A.shape[0]
    at, mine = _padded(s, rows)
    got = torch.bmm(_by_expert(A, at), W.float())
    whole = torch.cat([s["out"], s["out"].new_zeros(1, s["out"].shape[1])])
    whole[at] = got.to(s["type"])
    s["out"].copy_(whole[:rows])
    return s["out"]


def _plain(s):
    op = s["op"]
    if op == "clip":
        total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
        norm = total.sqrt()
        scale = (s["max_norm"] / norm).clamp(max=1.0).float()
        for g, o in zip(s["grads"], s["out"]):
            o.copy_(g.float() * scale)
        return norm.float(), s["flat_out"]
    if op == "quantize":
        _, value, scale = _mx_plain(s["X"], s["format"])
        return value.to(s["X"].dtype), scale
    if op == "forward":
        return _products(s, s["X"], s["W"].transpose(1, 2))
    if op == "dgrad":
        return _products(s, s["dY"], s["W"])
    if op == "mx_forward":
        return _products(s, _mx_plain(s["X"], "mxfp4")[1], _mx_values(s["Wc"], s["Ws"]).transpose(1, 2))
    at, _ = _padded(s, s["X"].shape[0])
    s["out"].copy_(torch.bmm(_by_expert(s["dY"], at).transpose(1, 2), _by_expert(s["X"], at)))
    return s["out"]


# ------------------------------------------------------------------- one pass

def run(s):
    if not own:
        return _plain(s)
    from expert_routed_ffn_gb300 import capi
    op = s["op"]
    if op == "clip":
        # into other tensors: a pass in place would leave nothing to clip for the next one
        return capi.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"]), s["flat_out"]
    if op == "quantize":
        codes, scales = capi.mx_quantize(s["X"], s["format"])
        return capi.mx_dequantize(codes, scales, s["format"], s["X"].dtype), scales
    if op == "forward":
        return capi.grouped_forward(s["X"], s["W"], s["offs"], out=s["out"])
    if op == "dgrad":
        return capi.grouped_dgrad(s["dY"], s["W"], s["offs"], out=s["out"])
    if op == "wgrad":
        return capi.grouped_wgrad(s["dY"], s["X"], s["offs"], out=s["out"])
    codes, scales = capi.mx_quantize(s["X"], "mxfp4")
    return capi.mx_grouped_forward(codes, scales, s["Wc"], s["Ws"], s["offs"], out=s["out"])


# ------------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "clip":
        square = 0.0
        for g in s["flat"]:
            for j in range(0, g.numel(), 1 << 26):
                square += float((g[j:j + (1 << 26)].double() ** 2).sum())
        norm = math.sqrt(square)
        return torch.tensor(norm, dtype=torch.float64), [g.double() * min(1.0, s["max_norm"] / norm) for g in s["flat"]]
    if op == "quantize":
        got = [_mx_exact(x, s["format"]) for x in s["X"]]
        return torch.stack([g[0] for g in got]), None
    offs = s["offs"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
    for e in range(case["E"]):
        r = slice(offs[e], offs[e + 1])
        if op == "wgrad":
            out[e] = s["dY"][r].double().t() @ s["X"][r].double()
        elif op == "mx_forward":
            w = torch.tensor([(c if c < 8 else c - 8) for c in range(16)], device=DEVICE)
            w = torch.tensor(E2M1, dtype=torch.float64, device=DEVICE)[w] * (1 - 2 * (torch.arange(16, device=DEVICE) > 7).double())
            codes = s["Wc"][e].long()
            values = torch.empty(case["N"], case["K"], dtype=torch.float64, device=DEVICE)
            values[:, 0::2], values[:, 1::2] = w[codes % 16], w[codes // 16]
            values *= torch.pow(2.0, s["Ws"][e].double() - 127).t().repeat_interleave(32, 1)
            out[r] = _mx_exact(s["X"][r], "mxfp4")[0] @ values.t()
        else:
            A = (s["X"] if op == "forward" else s["dY"])[r].double()
            W = s["W"][e].double()
            out[r] = A @ (W.t() if op == "forward" else W)
    return out


def _mx_exact(X, fmt):
    """The values of a tensor's codes from the definition: the spacing of the element
    type's values around each element, to nearest, ties to the even multiple."""
    x = X.double().unflatten(-1, (X.shape[-1] // 32, 32))
    bits, emax, low, most = (1, 2, 0, 6.0) if fmt == "mxfp4" else (3, 8, -6, 448.0)
    amax = x.abs().amax(-1, keepdim=True)
    shared = torch.floor(torch.log2(amax.clamp(min=1e-300))).clamp(min=-127 + emax) - emax
    v = x / torch.pow(2.0, shared)
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=1e-300))).clamp(min=low) - bits)
    v = (torch.round(v / step) * step).clamp(-most, most)
    return (v * torch.pow(2.0, shared)).reshape(X.shape), None
