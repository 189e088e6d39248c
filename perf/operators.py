"""The router and expert operators as they are measured.

Five operators around the dispatch and combine:

* ``gate``: router logits to the top-k expert ids and their weights;
* ``balance``: the load-balance loss with the per-expert counts and mean
  probabilities it is made of;
* ``gate_backward``: the gradient of weights and loss with respect to the
  logits;
* ``linear``: the experts' product over an expert-major buffer, with bias,
  activation and residual;
* ``linear_backward``: its gradients.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, by this package's calls.
"""

import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", torch.cuda.current_device())
else:
    DEV = torch.device("cpu")

ACTS = ("none", "gelu", "silu", "silu_glu")
SEGMENT = 128  # expert segments are padded to multiples of this many rows
BLOCK = 128    # columns (and weight rows) that share one E4M3 scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    def gate(name, **kw):
        return {"name": name, "op": "gate", **kw}

    def linear(name, op="linear", **kw):
        base = {"tokens": 16, "k": 8, "experts": 64, "in_dim": 7168, "out_dim": 2048, "act": "none",
                "bias": False, "residual": False, "fp8": False}
        return {"name": name, "op": op, **{**base, **kw}}

    return [
        # one token being answered: latency of a single launch
        gate("gate, one token", score="softmax", dtype="float32", tokens=1, experts=256, k=8,
             normalize=True, scale=1.0),
        # a long prompt batch of a bias-corrected sigmoid router
        gate("gate, prompts", score="sigmoid", dtype="bfloat16", tokens=16384, experts=256, k=8,
             normalize=True, scale=2.5),
        # a training step's batch (the prefill shape), every row valid
        {"name": "balance, training batch", "op": "balance", "score": "softmax",
         "dtype": "float32", "tokens": 4096, "experts": 256, "k": 8, "padding": 0},
        # a small padded batch, sizes that fill no wave
        {"name": "balance, padded batch", "op": "balance", "score": "sigmoid",
         "dtype": "bfloat16", "tokens": 1021, "experts": 60, "k": 4, "padding": 100},
        # gradient of both router outputs for the training batch
        {"name": "gate backward, training batch", "op": "gate_backward", "score": "softmax",
         "dtype": "float32", "tokens": 4096, "experts": 256, "k": 8, "normalize": True,
         "scale": 1.0, "padding": 0},
        # the same for many tokens over fewer experts, padded, bf16 logits
        {"name": "gate backward, padded batch", "op": "gate_backward", "score": "sigmoid",
         "dtype": "bfloat16", "tokens": 30011, "experts": 60, "k": 4, "normalize": False,
         "scale": 1.0, "padding": 512},
        # 16 sequences answering: two rows an expert, bound by the weights
        linear("experts, decode", act="silu_glu"),
        # a prefill batch over the experts of one rank: gate and up projection
        linear("experts, prefill", tokens=4096, experts=32, act="silu_glu"),
        # the same from an FP8 dispatch
        linear("experts, prefill FP8", tokens=4096, experts=32, act="silu_glu", fp8=True),
        # one shared expert over a ragged batch, everything in the epilogue
        linear("shared expert, ragged", tokens=1003, k=1, experts=1, in_dim=2048, out_dim=7168,
               act="gelu", bias=True, residual=True),
        # a training step's expert gradients
        linear("experts backward, training", op="linear_backward", tokens=2048, experts=32,
               act="silu_glu"),
        # a few experts of odd sizes with a bias
        linear("experts backward, ragged", op="linear_backward", tokens=301, k=2, experts=5,
               in_dim=1048, out_dim=520, act="none", bias=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(rng, lo, hi, step):
    return max(1, _log_int(rng, lo, hi) // step) * step


def draw(rng):
    op = rng.choice(("gate", "balance", "gate_backward", "linear", "linear", "linear_backward"))
    if op in ("gate", "balance", "gate_backward"):
        experts = _log_int(rng, 8, 512)
        case = {"op": op, "score": rng.choice(("softmax", "sigmoid")),
                "dtype": rng.choice(("float32", "bfloat16")), "experts": experts,
                "tokens": _log_int(rng, 1, 16384), "k": min(experts, rng.randint(1, 10))}
        if op != "balance":
            case["normalize"] = rng.random() < 0.6
            case["scale"] = rng.choice((1.0, 2.5))
        if op != "gate":
            case["padding"] = rng.randint(0, case["tokens"] // 4)
        return case
    experts = _log_int(rng, 1, 64)
    k = min(experts, rng.randint(1, 8))
    fp8 = op == "linear" and rng.random() < 0.4
    step = BLOCK if fp8 else 8
    act = rng.choice(ACTS)
    case = {"op": op, "tokens": _log_int(rng, 1, 2048), "k": k, "experts": experts,
            "in_dim": _odd(rng, 128, 7168, step), "out_dim": _odd(rng, 128, 2048, step),
            "act": act, "bias": rng.random() < 0.5,
            "residual": op == "linear" and rng.random() < 0.4, "fp8": fp8}
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=dtype) * scale) if scale != 1.0 else \
        torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _top(values, k):
    """The k largest of each row, ties to the lowest column."""
    return torch.sort(values, dim=-1, descending=True, stable=True)[1][:, :k]


def _prepare_router(case, g):
    T, E, k = case["tokens"], case["experts"], case["k"]
    dtype = getattr(torch, case["dtype"])
    logits = _normal(g, (T, E), torch.float32, 1.5).to(dtype)
    s = {"op": case["op"], "case": case, "logits": logits, "T": T, "E": E, "k": k,
         "sigmoid": case["score"] == "sigmoid", "normalize": case.get("normalize", False),
         "scale": case.get("scale", 1.0), "coef": 0.01}
    if case["op"] == "gate":
        s["bias"] = _normal(g, (E,), torch.float32, 0.1) if s["sigmoid"] else None
        s["indices"] = torch.zeros((T, k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.zeros((T, k), dtype=torch.float32, device=DEV)
    else:
        s["indices"] = _top(logits, k).to(torch.int32)
        s["mask"] = None
        if case["padding"]:  # the batch's last rows are padding
            s["mask"] = (torch.arange(T, device=DEV) < T - case["padding"]).to(torch.uint8)
        # per-expert counts and, last, the tokens that count
        valid = torch.ones(T, device=DEV, dtype=torch.int64) if s["mask"] is None else \
            s["mask"].to(torch.int64)
        counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
        counts.index_add_(0, s["indices"].reshape(-1).long(), valid.repeat_interleave(k))
        counts[E] = valid.sum()
        s["counts"] = counts.to(torch.int32)
        if case["op"] == "balance":
            s["out_counts"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
            s["prob_mean"] = torch.zeros(E, dtype=torch.float32, device=DEV)
            s["loss"] = torch.zeros(1, dtype=torch.float32, device=DEV)
        else:
            s["grad_weights"] = _normal(g, (T, k), torch.float32, 1e-3)
            s["grad_loss"] = torch.ones(1, dtype=torch.float32, device=DEV)
            s["grad_logits"] = torch.zeros((T, E), dtype=dtype, device=DEV)
    if own:
        import combine_mep_plan_amd as M
        s["cfg"] = M.MepGateConfig(E, k, M.MEP_SCORE_SIGMOID if s["sigmoid"] else M.MEP_SCORE_SOFTMAX,
                                   M.MEP_BF16 if dtype == torch.bfloat16 else M.MEP_FP32,
                                   int(s["normalize"]), s["scale"], s["coef"])
        if case["op"] == "balance":
            s["workspace"] = torch.zeros(M.mep_balance_workspace_bytes(s["cfg"], T),
                                         dtype=torch.uint8, device=DEV)
    return s


def _prepare_linear(case, g):
    T, k, E, K, N = (case[n] for n in ("tokens", "k", "experts", "in_dim", "out_dim"))
    rows, cap = T * k, T * k + 127 * E
    Nz = 2 * N if case["act"] == "silu_glu" else N
    # routing: k distinct experts a token; segments padded to whole blocks of rows
    picked = torch.rand((T, E), generator=g, device=DEV).argsort(dim=1)[:, :k]
    counts = torch.bincount(picked.reshape(-1), minlength=E)
    padded = (counts + SEGMENT - 1) // SEGMENT * SEGMENT
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = padded.cumsum(0)
    s = {"op": case["op"], "case": case, "E": E, "K": K, "N": N, "Nz": Nz, "rows": rows,
         "cap": cap, "act": case["act"], "most": int(counts.max()),
         "counts": counts.to(torch.int32), "offsets": offsets.to(torch.int32)}
    x = _normal(g, (cap, K), torch.bfloat16)
    w = _normal(g, (E, Nz, K), torch.bfloat16, 1.0 / math.sqrt(K))
    s["x_scales"] = s["w_scales"] = None
    if case["fp8"]:  # codes over their whole range, and scales as an absolute maximum gives them
        f8 = torch.float8_e4m3fn
        x, w = (x * 112).to(f8), (w * (112 * math.sqrt(K))).to(f8)
        s["x_scales"] = (torch.rand((cap, K // BLOCK), generator=g, device=DEV) + 0.5) / 112
        s["w_scales"] = (torch.rand((E, Nz // BLOCK, K // BLOCK), generator=g, device=DEV) + 0.5) \
            / (112 * math.sqrt(K))
    s["x"], s["w"] = x, w
    s["bias"] = _normal(g, (E, Nz), torch.float32, 0.1) if case["bias"] else None
    s["residual"] = _normal(g, (cap, N), torch.bfloat16) if case["residual"] else None
    if case["op"] == "linear":
        s["y"] = torch.zeros((cap, N), dtype=torch.bfloat16, device=DEV)
    else:
        s["grad_y"] = _normal(g, (cap, N), torch.bfloat16)
        # the product before the activation, as the forward pass keeps it
        s["z"] = _normal(g, (cap, Nz), torch.bfloat16) if case["act"] != "none" else None
        s["grad_x"] = torch.zeros((cap, K), dtype=torch.bfloat16, device=DEV)
        s["grad_w"] = torch.zeros((E, Nz, K), dtype=torch.bfloat16, device=DEV)
        s["grad_bias"] = torch.zeros((E, Nz), dtype=torch.float32, device=DEV) if case["bias"] else None
    if own:
        import combine_mep_plan_amd as M
        act = {"none": M.MEP_ACT_NONE, "gelu": M.MEP_ACT_GELU, "silu": M.MEP_ACT_SILU,
               "silu_glu": M.MEP_ACT_SILU_GLU}[case["act"]]
        s["cfg"] = M.MepLinearConfig(E, K, N, act, M.MEP_QUANT_FP8_E4M3_BLOCK128 if case["fp8"]
                                     else M.MEP_QUANT_NONE)
        if case["op"] == "linear_backward":
            s["workspace"] = torch.zeros(M.mep_linear_workspace_bytes(s["cfg"], cap),
                                         dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] in ("gate", "balance", "gate_backward"):
        return _prepare_router(case, g)
    return _prepare_linear(case, g)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(s):
    import combine_mep_plan_amd as M
    op = s["op"]
    if op == "gate":
        M.mep_gate(s["cfg"], s["logits"], s["bias"], s["T"], s["indices"], s["weights"])
        return s["indices"], s["weights"]
    if op == "balance":
        M.mep_balance_loss(s["cfg"], s["logits"], s["indices"], s["mask"], s["T"], s["out_counts"],
                           s["prob_mean"], s["loss"], s["workspace"])
        return s["out_counts"], s["prob_mean"], s["loss"]
    if op == "gate_backward":
        M.mep_gate_backward(s["cfg"], s["logits"], s["indices"], s["mask"], s["T"],
                            s["grad_weights"], s["counts"], s["grad_loss"], s["grad_logits"])
        return s["grad_logits"]
    if op == "linear":
        M.mep_expert_linear(s["cfg"], s["x"], s["x_scales"], s["counts"], s["offsets"], s["cap"],
                            s["rows"], s["w"], s["w_scales"], s["bias"], s["residual"], s["y"],
                            None)
        return s["y"]
    M.mep_expert_linear_backward(s["cfg"], s["grad_y"], s["z"], s["x"], s["w"], s["counts"],
                                 s["offsets"], s["cap"], s["rows"], s["grad_x"], s["grad_w"],
                                 s["grad_bias"], s["workspace"])
    return s["grad_x"], s["grad_w"], s["grad_bias"]


def _softmax(x):
    z = torch.exp(x - x.amax(dim=-1, keepdim=True))
    return z / z.sum(dim=-1, keepdim=True)


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _run_gate(s):
    x = s["logits"].float()
    if s["sigmoid"]:
        # the order of the scores in 64 bits: neighbours may be closer than 32 bits tell
        idx = _top(_sigmoid(x.double()) + s["bias"].double(), s["k"])
        v = _sigmoid(x).gather(1, idx)
    else:
        idx = _top(x, s["k"])
        v = _softmax(x).gather(1, idx)
    if s["normalize"]:
        v = v / v.sum(dim=-1, keepdim=True)
    return idx.to(torch.int32), v * s["scale"]


def _probabilities(s, x):
    if not s["sigmoid"]:
        return _softmax(x)
    v = _sigmoid(x)
    return v / v.sum(dim=-1, keepdim=True)


def _run_balance(s):
    p, E, k = _probabilities(s, s["logits"].float()), s["E"], s["k"]
    hits = torch.zeros_like(p).scatter_add_(1, s["indices"].long(),
                                            torch.ones_like(s["indices"], dtype=torch.float32))
    if s["mask"] is None:
        n = torch.full((), s["T"], dtype=torch.float32, device=DEV)
    else:
        keep = s["mask"].bool()[:, None]
        p, hits = torch.where(keep, p, 0.0), torch.where(keep, hits, 0.0)
        n = s["mask"].float().sum()
    counts, mean = hits.sum(0), p.sum(0) / n
    loss = (counts * mean).sum() * (s["coef"] * E / k) / n
    return torch.cat([counts, n[None]]).to(torch.int32), mean, loss[None]


def _run_gate_backward(s):
    x, idx, gw = s["logits"].float(), s["indices"].long(), s["grad_weights"] * s["scale"]
    n = s["counts"][s["E"]].float()
    a = s["counts"][: s["E"]].float() * (s["grad_loss"] * (s["coef"] * s["E"] / s["k"]) / (n * n))
    grad = torch.zeros_like(x)
    p = _probabilities(s, x)
    tilt = a - (p * a).sum(-1, keepdim=True)
    if s["sigmoid"]:
        v = _sigmoid(x)
        slope = v * (1 - v)
        grad = slope / v.sum(-1, keepdim=True) * tilt
        vk, sk = v.gather(1, idx), slope.gather(1, idx)
        if s["normalize"]:
            total = vk.sum(-1, keepdim=True)
            gw = (gw - (gw * vk / total).sum(-1, keepdim=True)) / total
        grad.scatter_add_(1, idx, gw * sk)
    else:
        pk = p.gather(1, idx)
        grad = p * tilt
        if s["normalize"]:
            q = pk / pk.sum(-1, keepdim=True)
            grad.scatter_add_(1, idx, q * (gw - (gw * q).sum(-1, keepdim=True)))
        else:
            grad = grad - p * (gw * pk).sum(-1, keepdim=True)
            grad.scatter_add_(1, idx, gw * pk)
    if s["mask"] is not None:
        grad = torch.where(s["mask"].bool()[:, None], grad, 0.0)
    return grad.to(s["logits"].dtype)


def _rows(s):
    """The buffer row of each expert's i-th row [E, most]; the row past the buffer where it has none."""
    i = torch.arange(s["most"], device=DEV)
    at = s["offsets"][:-1, None].long() + i
    return torch.where(i < s["counts"][:, None], at, s["cap"])


def _take(buffer, rows, dtype):
    """The rows of a buffer by expert, zeros where there is none."""
    got = buffer[rows.clamp(max=buffer.shape[0] - 1)].to(dtype)
    return torch.where((rows < buffer.shape[0])[..., None], got, torch.zeros((), dtype=dtype, device=DEV))


def _put(rows, values, cap):
    """values [E, most, C] in the rows of a buffer of zeros."""
    out = torch.zeros((cap + 1, values.shape[-1]), dtype=values.dtype, device=DEV)
    out[rows.reshape(-1)] = values.reshape(-1, values.shape[-1])
    return out[:cap]


def _gelu(z):
    return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))


def _run_linear(s):
    rows = _rows(s)
    x, w = s["x"].float(), s["w"].float()
    if s["x_scales"] is not None:
        x = x * s["x_scales"].repeat_interleave(BLOCK, 1)
        w = w * s["w_scales"].repeat_interleave(BLOCK, 1).repeat_interleave(BLOCK, 2)
    z = torch.bmm(_take(x, rows, torch.float32), w.transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"][:, None]
    if s["act"] == "silu_glu":
        gate, up = z[..., : s["N"]], z[..., s["N"]:]
        y = gate * _sigmoid(gate) * up
    else:
        y = {"none": lambda v: v, "gelu": _gelu, "silu": lambda v: v * _sigmoid(v)}[s["act"]](z)
    if s["residual"] is not None:
        y = y + _take(s["residual"], rows, torch.float32)
    return _put(rows, y.to(torch.bfloat16), s["cap"])


def _grad_z(act, gy, z, N):
    """The gradient before the activation, in the type of its inputs."""
    if act == "none":
        return gy
    if act == "gelu":
        return gy * (0.5 * (1 + torch.erf(z / math.sqrt(2)))
                     + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    gate = z[..., :N]
    sig = _sigmoid(gate)
    slope = sig * (1 + gate * (1 - sig))
    if act == "silu":
        return gy * slope
    return torch.cat([gy * z[..., N:] * slope, gy * gate * sig], dim=-1)


def _run_linear_backward(s):
    rows = _rows(s)
    gy = _take(s["grad_y"], rows, torch.float32)
    z = None if s["z"] is None else _take(s["z"], rows, torch.float32)
    gz = _grad_z(s["act"], gy, z, s["N"])
    gx = torch.bmm(gz, s["w"].float())
    gw = torch.bmm(gz.transpose(1, 2), _take(s["x"], rows, torch.float32))
    gb = gz.sum(1) if s["bias"] is not None else None
    return _put(rows, gx.to(torch.bfloat16), s["cap"]), gw.to(torch.bfloat16), gb


def run(state):
    if own:
        return _run_own(state)
    return {"gate": _run_gate, "balance": _run_balance, "gate_backward": _run_gate_backward,
            "linear": _run_linear, "linear_backward": _run_linear_backward}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    T, k, E = case["tokens"], case["k"], case["experts"]
    if case["op"] in ("gate", "balance", "gate_backward"):
        size = 4 if case["dtype"] == "float32" else 2
        nbytes = T * E * size
        if case["op"] == "gate":
            nbytes += 8 * T * k + (4 * E if case["score"] == "sigmoid" else 0)
        elif case["op"] == "balance":
            nbytes += 4 * T * k + 8 * E + (T if case["padding"] else 0)
        else:
            nbytes += T * E * size + 8 * T * k + 4 * E + (T if case["padding"] else 0)
        return {"bytes": nbytes, "flops": 8 * T * E}
    rows, K, N = T * k, case["in_dim"], case["out_dim"]
    Nz = 2 * N if case["act"] == "silu_glu" else N
    used = E * (1 - (1 - k / E) ** T)  # experts that any token names, on average
    size = 1 if case["fp8"] else 2
    nbytes = size * (rows * K + used * Nz * K) + 2 * rows * N
    if case["fp8"]:
        nbytes += 4 * (rows * (K // BLOCK) + used * (Nz // BLOCK) * (K // BLOCK))
    nbytes += (4 * used * Nz if case["bias"] else 0) + (2 * rows * N if case["residual"] else 0)
    flops = 2 * rows * Nz * K
    if case["op"] == "linear_backward":
        nbytes += 2 * rows * K + 2 * E * Nz * K + (2 * rows * Nz if case["act"] != "none" else 0)
        flops *= 2
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_scores(case, logits):
    """Each token's scores and the probabilities made of them."""
    if case["score"] == "sigmoid":
        v = torch.sigmoid(logits)
        return v, v / v.sum(dim=1, keepdim=True)
    v = torch.softmax(logits, dim=1)
    return v, v


def _exact_gate(case, s):
    x = s["logits"].double()
    v, _ = _exact_scores(case, x)
    order = x if case["score"] == "softmax" else v + s["bias"].double()
    idx = torch.argsort(order, dim=1, descending=True, stable=True)[:, : case["k"]]
    w = torch.gather(v, 1, idx)
    if case["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), case["scale"] * w


def _valid(case):
    return case["tokens"] - case["padding"]


def _exact_balance(case, s):
    n, E, k = _valid(case), case["experts"], case["k"]
    _, p = _exact_scores(case, s["logits"][:n].double())
    counts = np.bincount(s["indices"][:n].cpu().numpy().reshape(-1), minlength=E)
    mean = p.mean(dim=0)
    share = torch.from_numpy(counts / (k * n)).to(DEV)
    loss = s["coef"] * E * torch.dot(share, mean)
    return (torch.from_numpy(np.append(counts, n).astype(np.int32)), mean, loss.reshape(1))


def _exact_gate_backward(case, s):
    """By differentiating the definitions."""
    n, E, k = _valid(case), case["experts"], case["k"]
    x = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        v, p = _exact_scores(case, x)
        w = torch.gather(v, 1, s["indices"].long())
        if case["normalize"]:
            w = w / w.sum(dim=1, keepdim=True)
        share = s["counts"][:E].double() / (k * n)
        loss = s["coef"] * E * torch.dot(share, p[:n].mean(dim=0))
        total = (case["scale"] * w[:n] * s["grad_weights"][:n].double()).sum() \
            + loss * s["grad_loss"].double()[0]
        (grad,) = torch.autograd.grad(total, x)
    return grad


def _exact_segments(s):
    counts, offsets = s["counts"].tolist(), s["offsets"].tolist()
    return [(e, offsets[e], offsets[e] + counts[e]) for e in range(len(counts)) if counts[e]]


def _exact_act(case, z):
    if case["act"] == "gelu":
        return torch.nn.functional.gelu(z)
    if case["act"] == "silu":
        return torch.nn.functional.silu(z)
    if case["act"] == "silu_glu":
        gate, up = z.chunk(2, dim=-1)
        return torch.nn.functional.silu(gate) * up
    return z


def _exact_linear(case, s):
    y = torch.zeros((s["cap"], s["N"]), dtype=torch.float64, device=DEV)
    for e, a, b in _exact_segments(s):
        x, w = s["x"][a:b].double(), s["w"][e].double()
        if case["fp8"]:
            x = (x.unflatten(1, (-1, BLOCK)) * s["x_scales"][a:b, :, None].double()).flatten(1)
            ws = s["w_scales"][e].double()
            w = w * torch.kron(ws, torch.ones((BLOCK, BLOCK), dtype=torch.float64, device=DEV))
        z = x @ w.T
        if case["bias"]:
            z = z + s["bias"][e].double()
        y[a:b] = _exact_act(case, z)
        if case["residual"]:
            y[a:b] += s["residual"][a:b].double()
    return y


def _exact_linear_backward(case, s):
    gx = torch.zeros((s["cap"], s["K"]), dtype=torch.float64, device=DEV)
    gw = torch.zeros((s["E"], s["Nz"], s["K"]), dtype=torch.float64, device=DEV)
    gb = torch.zeros((s["E"], s["Nz"]), dtype=torch.float64, device=DEV)
    for e, a, b in _exact_segments(s):
        gz = s["grad_y"][a:b].double()
        if case["act"] != "none":
            z = s["z"][a:b].double().requires_grad_(True)
            with torch.enable_grad():
                (gz,) = torch.autograd.grad(_exact_act(case, z), z, gz)
        gx[a:b] = gz @ s["w"][e].double()
        gw[e] = gz.T.contiguous() @ s["x"][a:b].double()
        gb[e] = gz.sum(0)
    return gx, gw, gb if case["bias"] else None


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "balance": _exact_balance, "gate_backward": _exact_gate_backward,
            "linear": _exact_linear, "linear_backward": _exact_linear_backward}[case["op"]](case, s)
