"""The operators around a mixture-of-experts block as they are measured.

Four operators:

* ``gate_grouped``: a router that first chooses groups of experts, then the
  experts inside them;
* ``norm``: what stands between two blocks: the norm of a block's output, its
  gate, the scaled residual, and the norm of the next block's input, which may
  leave as E4M3 codes for the dispatch;
* ``norm_backward``: its gradients;
* ``clip``: the global norm of a list of gradients, and the clipping by it.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, by this package's calls.
"""

import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", torch.cuda.current_device())
else:
    DEV = torch.device("cpu")

BLOCK = 128  # columns that share one E4M3 scale
EPS = 1e-6   # of the norms
GRAD = 1e-3  # size of a gradient's values


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm_case(name, op, **kw):
    base = {"dtype": "bfloat16", "tokens": 1, "hidden": 7168, "post": "none", "pre": "rms", "block": True,
            "gate": "none", "sigmoid": False, "bias": False, "residual_scale": 1.0, "block_scale": 1.0,
            "rows": True, "codes": False}
    return {"name": name, "op": op, **base, **kw}


def listed():
    return [
        # one token being answered by a router over 8 ranks' experts: latency of a launch
        {"name": "grouped gate, one token", "op": "gate_grouped", "score": "sigmoid", "group": "top2",
         "dtype": "float32", "tokens": 1, "experts": 256, "groups": 8, "top_groups": 4, "k": 8,
         "normalize": True, "scale": 2.5},
        # a long prompt batch of the same router
        {"name": "grouped gate, prompts", "op": "gate_grouped", "score": "sigmoid", "group": "top2",
         "dtype": "bfloat16", "tokens": 16384, "experts": 256, "groups": 8, "top_groups": 4, "k": 8,
         "normalize": True, "scale": 2.5},
        # a small batch of a softmax router, groups by their best expert, sizes that fill no lane
        {"name": "grouped gate, ragged", "op": "gate_grouped", "score": "softmax", "group": "max",
         "dtype": "float32", "tokens": 1021, "experts": 60, "groups": 6, "top_groups": 3, "k": 4,
         "normalize": False, "scale": 1.0},
        # one token being answered: the residual added, the next block's input normed
        _norm_case("norm, one token", "norm"),
        # 128 sequences answering, rows for an FP8 dispatch beside those for the router
        _norm_case("norm, decode", "norm", tokens=128, codes=True),
        # a prefill batch between two blocks that norm both ends of each, a token's
        # block output gated, rows for the router and codes for the dispatch
        _norm_case("norm, prefill", "norm", tokens=4096, post="rms", gate="token", sigmoid=True, codes=True),
        # a ragged fp32 batch, layer norms with biases, every element gated, residual scaled
        _norm_case("norm, ragged", "norm", dtype="float32", tokens=1003, hidden=2056, post="layer",
                   pre="layer", gate="element", bias=True, residual_scale=0.5, block_scale=1.5),
        # a training step's batch, gradients of rows, gate and both weights
        _norm_case("norm backward, training", "norm_backward", tokens=4096, post="rms", gate="token",
                   sigmoid=True),
        # gradients of the ragged form, smaller still
        _norm_case("norm backward, ragged", "norm_backward", dtype="float32", tokens=301, hidden=1048,
                   post="layer", pre="layer", gate="element", bias=True, residual_scale=0.5,
                   block_scale=1.5),
        # gradients of a layer's 32 experts, router and norms, into the optimizer's buffers
        {"name": "clip, experts", "op": "clip", "experts": 32, "in_dim": 7168, "out_dim": 2048, "small": 4,
         "clipped": True, "inplace": False},
        # many small tensors of odd sizes (biases, norms, routers' rows), which count by launches
        {"name": "clip, small tensors", "op": "clip", "experts": 1, "in_dim": 520, "out_dim": 264, "small": 56,
         "clipped": True, "inplace": False},
        # a settled training run's usual step: the norm is below the limit, gradients stay
        {"name": "clip, below the limit", "op": "clip", "experts": 4, "in_dim": 7168, "out_dim": 2048,
         "small": 20, "clipped": False, "inplace": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gate_grouped", "norm", "norm", "norm_backward", "clip"))
    if op == "gate_grouped":
        groups, size = rng.randint(2, 16), _log_int(rng, 2, 32)
        top = rng.randint(1, groups)
        return {"op": op, "score": rng.choice(("softmax", "sigmoid")), "group": rng.choice(("max", "top2")),
                "dtype": rng.choice(("float32", "bfloat16")), "tokens": _log_int(rng, 1, 16384),
                "experts": groups * size, "groups": groups, "top_groups": top,
                "k": rng.randint(1, min(10, top * size)), "normalize": rng.random() < 0.6,
                "scale": rng.choice((1.0, 2.5))}
    if op == "clip":
        return {"op": op, "experts": _log_int(rng, 1, 16), "in_dim": _log_int(rng, 16, 7168),
                "out_dim": _log_int(rng, 16, 2048), "small": rng.randint(0, 56),
                "clipped": rng.random() < 0.5, "inplace": False}
    codes = op == "norm" and rng.random() < 0.4
    step = BLOCK if codes else 8
    block = rng.random() < 0.8
    case = {"op": op, "dtype": rng.choice(("float32", "bfloat16")), "tokens": _log_int(rng, 1, 4096),
            "hidden": max(1, _log_int(rng, 128, 8192) // step) * step,
            "post": rng.choice(("none", "rms", "layer")) if block else "none",
            "pre": rng.choice(("rms", "layer")), "block": block,
            "gate": rng.choice(("none", "token", "element")) if block else "none",
            "sigmoid": rng.random() < 0.5, "bias": rng.random() < 0.4,
            "residual_scale": rng.choice((1.0, 0.5)) if block else 1.0,
            "block_scale": rng.choice((1.0, 0.22)) if block else 1.0,
            "rows": not codes or rng.random() < 0.5, "codes": codes}
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return t if scale == 1.0 else t.mul_(scale)


def _prepare_gate(case, g):
    T, E, k = case["tokens"], case["experts"], case["k"]
    dtype = getattr(torch, case["dtype"])
    s = {"case": case, "logits": _normal(g, (T, E), torch.float32, 1.5).to(dtype),
         "bias": _normal(g, (E,), torch.float32, 0.1) if case["score"] == "sigmoid" else None,
         "indices": torch.zeros((T, k), dtype=torch.int32, device=DEV),
         "weights": torch.zeros((T, k), dtype=torch.float32, device=DEV)}
    if own:
        import combine_mep_plan_amd as M
        s["cfg"] = M.MepGateConfig(
            E, k, M.MEP_SCORE_SIGMOID if case["score"] == "sigmoid" else M.MEP_SCORE_SOFTMAX,
            M.MEP_BF16 if dtype == torch.bfloat16 else M.MEP_FP32, int(case["normalize"]), case["scale"], 0.0)
        s["by"] = M.MEP_GROUP_TOP2 if case["group"] == "top2" else M.MEP_GROUP_MAX
    return s


def _gate_values(case, g, dtype):
    if case["gate"] == "token":
        return _normal(g, (case["tokens"],))
    if case["gate"] == "element":
        return _normal(g, (case["tokens"], case["hidden"]), dtype)
    return None


def _prepare_norm(case, g):
    T, H = case["tokens"], case["hidden"]
    dtype = getattr(torch, case["dtype"])
    backward = case["op"] == "norm_backward"
    rows = lambda: torch.zeros((T, H), dtype=dtype, device=DEV)  # noqa: E731
    columns = lambda on: torch.zeros(H, device=DEV) if on else None  # noqa: E731
    block, post, biased = case["block"], case["post"] != "none", case["bias"]
    s = {"case": case, "T": T,
         # a stream whose rows differ in size, as they do along the depth of a model
         "x": (_normal(g, (T, H)) * (_normal(g, (T, 1)).abs() + 0.5)).to(dtype),
         "y": _normal(g, (T, H), dtype) if block else None,
         "gate": _gate_values(case, g, dtype),
         "post_weight": 1 + _normal(g, (H,), scale=0.1) if post else None,
         "post_bias": _normal(g, (H,), scale=0.1) if post and biased else None,
         "pre_weight": 1 + _normal(g, (H,), scale=0.1),
         "pre_bias": _normal(g, (H,), scale=0.1) if biased else None}
    if backward:
        s["grad_s"], s["grad_n"] = _normal(g, (T, H), dtype), _normal(g, (T, H), dtype)
        s["grad_x"], s["grad_y"] = rows(), rows() if block else None
        s["grad_gate"] = None if s["gate"] is None else torch.zeros_like(s["gate"])
        s["columns"] = [columns(post), columns(post and biased), columns(True), columns(biased)]
    else:
        s["s"] = rows() if block else None
        s["n"] = rows() if case["rows"] else None
        s["codes"] = s["scales"] = None
        if case["codes"]:
            s["codes"] = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device=DEV)
            s["scales"] = torch.zeros((T, H // BLOCK), device=DEV)
    if own:
        import combine_mep_plan_amd as M
        kinds = {"none": M.MEP_NORM_NONE, "rms": M.MEP_NORM_RMS, "layer": M.MEP_NORM_LAYER}
        s["cfg"] = M.MepNormConfig(
            H, M.MEP_BF16 if dtype == torch.bfloat16 else M.MEP_FP32, kinds[case["post"]], kinds[case["pre"]],
            {"none": M.MEP_BLOCK_GATE_NONE, "token": M.MEP_BLOCK_GATE_TOKEN,
             "element": M.MEP_BLOCK_GATE_ELEMENT}[case["gate"]],
            int(case["sigmoid"]), EPS, 0.0, case["residual_scale"], case["block_scale"])
        if backward:
            s["workspace"] = torch.zeros(M.mep_block_norm_workspace_bytes(s["cfg"], T), dtype=torch.uint8,
                                         device=DEV)
    return s


def _shapes(case):
    """(shape, type) of each gradient: the experts' two weights, the router's, then
    vectors of ragged lengths, every other one in fp32."""
    E, K, N = case["experts"], case["in_dim"], case["out_dim"]
    vectors = [((K + 37 * i + i % 3,), "float32" if i % 2 else "bfloat16") for i in range(case["small"])]
    return [((E, 2 * N, K), "bfloat16"), ((E, K, N), "bfloat16"), ((E, K), "float32"), *vectors]


def _numel(case):
    return sum(math.prod(shape) for shape, _ in _shapes(case))


def _prepare_clip(case, g):
    grads = [_normal(g, shape, getattr(torch, dtype), GRAD) for shape, dtype in _shapes(case)]
    expected = GRAD * math.sqrt(_numel(case))
    s = {"case": case, "grads": grads, "max_norm": expected * (0.3 if case["clipped"] else 2.0),
         "out": grads if case["inplace"] else [torch.zeros_like(t) for t in grads],
         "norm": torch.zeros(1, device=DEV)}
    if own:
        import combine_mep_plan_amd as M
        s["list"] = M.MepGrads(grads, s["out"])
        s["workspace"] = torch.zeros(M.mep_grad_workspace_bytes(s["list"]), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "gate_grouped":
        return _prepare_gate(case, g)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    return _prepare_norm(case, g)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(s):
    import combine_mep_plan_amd as M
    case = s["case"]
    if case["op"] == "gate_grouped":
        M.mep_gate_grouped(s["cfg"], case["groups"], case["top_groups"], s["by"], s["logits"], s["bias"],
                           case["tokens"], s["indices"], s["weights"])
        return s["indices"], s["weights"]
    if case["op"] == "norm":
        M.mep_block_norm(s["cfg"], s["x"], s["y"], s["gate"], s["post_weight"], s["post_bias"],
                         s["pre_weight"], s["pre_bias"], s["T"], s["s"], s["n"], s["codes"], s["scales"])
        return s["s"], s["n"], s["codes"], s["scales"]
    if case["op"] == "norm_backward":
        # x stands for the stream that the forward pass left
        M.mep_block_norm_backward(s["cfg"], s["grad_s"], s["grad_n"], s["x"], s["y"], s["gate"],
                                  s["post_weight"], s["post_bias"], s["pre_weight"], s["T"], s["grad_x"],
                                  s["grad_y"], s["grad_gate"], *s["columns"], s["workspace"])
        return s["grad_x"], s["grad_y"], s["grad_gate"], *s["columns"]
    M.mep_grad_norm(s["list"], s["norm"], s["workspace"])
    M.mep_grad_clip(s["list"], s["norm"], s["max_norm"])
    return s["norm"], *s["out"]


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _softmax(x):
    z = torch.exp(x - x.amax(dim=-1, keepdim=True))
    return z / z.sum(dim=-1, keepdim=True)


def _best(values, n):
    """The n largest of each row, ties to the lowest column."""
    return torch.sort(values, dim=-1, descending=True, stable=True)[1][:, :n]


def _run_gate(s):
    case, x = s["case"], s["logits"].float()
    T, E, G = case["tokens"], case["experts"], case["groups"]
    # orders in 64 bits: neighbours may be closer than 32 bits tell
    if case["score"] == "sigmoid":
        order = _sigmoid(x.double()) + s["bias"].double()
        value = _sigmoid(x)
    else:
        order = _softmax(x.double())
        value = _softmax(x)
    inside = torch.sort(order.reshape(T, G, E // G), dim=-1, descending=True)[0]
    score = inside[..., 0] + inside[..., 1] if case["group"] == "top2" else inside[..., 0]
    kept = torch.zeros((T, G), dtype=torch.bool, device=DEV)
    kept.scatter_(1, _best(score, case["top_groups"]), True)
    idx = _best(torch.where(kept.repeat_interleave(E // G, 1), order, -math.inf), case["k"])
    v = value.gather(1, idx)
    if case["normalize"]:
        v = v / v.sum(dim=-1, keepdim=True)
    return idx.to(torch.int32), v * case["scale"]


def _hat(kind, u):
    """(normed rows, the factor that normed them)."""
    if kind == "none":
        return u, torch.ones((), device=DEV)
    if kind == "layer":
        u = u - u.mean(dim=-1, keepdim=True)
    r = 1 / torch.sqrt((u * u).mean(dim=-1, keepdim=True) + EPS)
    return u * r, r


def _affine(u, weight, bias):
    u = u if weight is None else u * weight
    return u if bias is None else u + bias


def _open(s):
    """The gate as a factor of rows, and its slope."""
    if s["gate"] is None:
        one = torch.ones((), device=DEV)
        return one, one
    g = s["gate"].float()
    g = g[:, None] if g.dim() == 1 else g
    if not s["case"]["sigmoid"]:
        return g, torch.ones_like(g)
    g = _sigmoid(g)
    return g, g * (1 - g)


def _run_norm(s):
    case, dtype = s["case"], s["x"].dtype
    u = s["x"].float() * case["residual_scale"]
    out = None
    if case["block"]:
        v = _affine(_hat(case["post"], s["y"].float())[0], s["post_weight"], s["post_bias"])
        u = u + v * _open(s)[0] * case["block_scale"]
        out = u.to(dtype)
    n = _affine(_hat(case["pre"], u)[0], s["pre_weight"], s["pre_bias"])
    codes = scales = None
    if case["codes"]:
        blocks = n.reshape(n.shape[0], -1, BLOCK)
        scales = blocks.abs().amax(dim=-1) / 448
        codes = (blocks / torch.where(scales == 0, 1.0, scales)[..., None]).reshape(n.shape)
        codes = codes.to(torch.float8_e4m3fn)
    return out, n.to(dtype) if case["rows"] else None, codes, scales


def _hat_backward(kind, hat, r, grad):
    if kind == "none":
        return grad
    grad_in = grad - hat * (grad * hat).mean(dim=-1, keepdim=True)
    if kind == "layer":
        grad_in = grad_in - grad.mean(dim=-1, keepdim=True)
    return grad_in * r


def _run_norm_backward(s):
    case, dtype = s["case"], s["x"].dtype
    grad_n = s["grad_n"].float()
    hat, r = _hat(case["pre"], s["x"].float())
    grad = s["grad_s"].float() + _hat_backward(case["pre"], hat, r, grad_n * s["pre_weight"])
    grad_x = (grad * case["residual_scale"]).to(dtype)
    pre_w, pre_b = (grad_n * hat).sum(0), grad_n.sum(0) if case["bias"] else None
    if not case["block"]:
        return grad_x, None, None, None, None, pre_w, pre_b
    hat, r = _hat(case["post"], s["y"].float())
    v = _affine(hat, s["post_weight"], s["post_bias"])
    g, slope = _open(s)
    grad_gate = None
    if s["gate"] is not None:
        grad_gate = grad * v * case["block_scale"]
        if s["gate"].dim() == 1:
            grad_gate = grad_gate.sum(-1, keepdim=True)
        grad_gate = (grad_gate * slope).reshape(s["gate"].shape).to(s["gate"].dtype)
    grad_v = grad * g * case["block_scale"]
    post_w = (grad_v * hat).sum(0) if s["post_weight"] is not None else None
    post_b = grad_v.sum(0) if s["post_bias"] is not None else None
    if s["post_weight"] is not None:
        grad_v = grad_v * s["post_weight"]
    return grad_x, _hat_backward(case["post"], hat, r, grad_v).to(dtype), grad_gate, post_w, post_b, pre_w, pre_b


def _run_clip(s):
    squares = [t.float().square().sum() for t in s["grads"]]
    norm = torch.stack(squares).double().sum().sqrt().float()
    factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return norm[None], *[(t.float() * factor).to(t.dtype) for t in s["grads"]]


def run(state):
    if own:
        return _run_own(state)
    return {"gate_grouped": _run_gate, "norm": _run_norm, "norm_backward": _run_norm_backward,
            "clip": _run_clip}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "clip":
        nbytes = sum(math.prod(shape) * (4 if dtype == "float32" else 2) for shape, dtype in _shapes(case))
        # read for the norm; read again and written where the gradients change or move
        return {"bytes": nbytes if case["inplace"] and not case["clipped"] else 3 * nbytes,
                "flops": 3 * _numel(case)}
    T, size = case["tokens"], 4 if case["dtype"] == "float32" else 2
    if case["op"] == "gate_grouped":
        E = case["experts"]
        return {"bytes": T * E * size + 8 * T * case["k"] + (4 * E if case["score"] == "sigmoid" else 0),
                "flops": 10 * T * E}
    H = case["hidden"]
    row, vectors = T * H * size, 4 * H
    gate = {"none": 0, "token": 4 * T, "element": row}[case["gate"]]
    block, post = case["block"], case["post"] != "none"
    weights = (1 + post) * (1 + case["bias"]) * vectors
    if case["op"] == "norm":
        nbytes = row * (3 if block else 1) + gate + weights + (row if case["rows"] else 0)
        if case["codes"]:
            nbytes += T * H + 4 * T * (H // BLOCK)
        return {"bytes": nbytes, "flops": 16 * T * H}
    # grad_s, grad_n, the stream and the block's output in; their gradients out
    nbytes = row * (6 if block else 4) + 2 * gate + 2 * weights
    return {"bytes": nbytes, "flops": 32 * T * H}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_gate(case, s):
    x = s["logits"].double()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(x)
        q = p + s["bias"].double()
    else:
        p = q = torch.softmax(x, dim=1)
    groups = q.unflatten(1, (case["groups"], -1))
    of_group = groups.topk(2 if case["group"] == "top2" else 1, dim=2)[0].sum(2)
    # a group's rank: how many come before it
    g = torch.arange(case["groups"], device=DEV)
    before = (of_group[:, None] > of_group[:, :, None]) | \
        ((of_group[:, None] == of_group[:, :, None]) & (g[None, None] < g[None, :, None]))
    dropped = before.sum(2) >= case["top_groups"]
    q = groups.masked_fill(dropped[..., None], -math.inf).flatten(1)
    idx = torch.argsort(q, dim=1, descending=True, stable=True)[:, : case["k"]]
    w = torch.gather(p, 1, idx)
    if case["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), case["scale"] * w


def _exact_one(case, kind, u, weight, bias):
    H = (case["hidden"],)
    if kind == "layer":
        return torch.nn.functional.layer_norm(u, H, weight, bias, EPS)
    if kind == "rms":
        u = u * torch.rsqrt(u.pow(2).mean(-1, keepdim=True) + EPS)
    u = u if weight is None else u * weight
    return u if bias is None else u + bias


def _exact_stream(case, x, y, gate, weight, bias):
    if y is None:
        return case["residual_scale"] * x
    v = _exact_one(case, case["post"], y, weight, bias)
    if gate is not None:
        g = torch.sigmoid(gate) if case["sigmoid"] else gate
        v = v * (g.unsqueeze(1) if g.dim() == 1 else g)
    return case["residual_scale"] * x + case["block_scale"] * v


def _double(t):
    return None if t is None else t.double()


def _exact_norm(case, s):
    d = {k: _double(s[k]) for k in ("x", "y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")}
    u = _exact_stream(case, d["x"], d["y"], d["gate"], d["post_weight"], d["post_bias"])
    n = _exact_one(case, case["pre"], u, d["pre_weight"], d["pre_bias"])
    codes = scales = None
    if case["codes"]:  # before their rounding
        b = n.unflatten(1, (-1, BLOCK))
        scales = b.abs().max(dim=2)[0] / 448
        codes = (b / scales.clamp_min(1e-300)[..., None]).flatten(1)
    return u if case["block"] else None, n if case["rows"] else None, codes, scales


def _exact_norm_backward(case, s):
    """By differentiating the definitions: the next norm at the stream that is given, the
    block's part at the block's output."""
    names = ("y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")
    d = {k: None if s[k] is None else s[k].double().requires_grad_(True) for k in names}
    stream = s["x"].double().requires_grad_(True)
    with torch.enable_grad():
        n = _exact_one(case, case["pre"], stream, d["pre_weight"], d["pre_bias"])
        asked = [t for t in (d["pre_weight"], d["pre_bias"]) if t is not None]
        got = torch.autograd.grad(n, [stream] + asked, s["grad_n"].double())
    pre = dict(zip([k for k in ("pre_weight", "pre_bias") if d[k] is not None], got[1:]))
    total = s["grad_s"].double() + got[0]
    x = torch.zeros_like(stream).detach().requires_grad_(True)
    with torch.enable_grad():
        u = _exact_stream(case, x, d["y"], d["gate"], d["post_weight"], d["post_bias"])
        asked = ["x"] + [k for k in ("y", "gate", "post_weight", "post_bias") if d[k] is not None]
        got = dict(zip(asked, torch.autograd.grad(u, [x] + [d[k] for k in asked[1:]], total)))
    return (got["x"], got.get("y"), got.get("gate"), got.get("post_weight"), got.get("post_bias"),
            pre["pre_weight"], pre.get("pre_bias"))


def _exact_clip(case, s):
    pieces = [p for t in s["grads"] for p in t.reshape(-1).split(1 << 27)]
    norm = torch.zeros((), dtype=torch.float64, device=DEV)
    for p in pieces:
        norm = torch.hypot(norm, torch.linalg.vector_norm(p.double()))
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return norm.reshape(1), *[t.double().mul_(factor) for t in s["grads"]]


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate_grouped": _exact_gate, "norm": _exact_norm, "norm_backward": _exact_norm_backward,
            "clip": _exact_clip}[case["op"]](case, s)
