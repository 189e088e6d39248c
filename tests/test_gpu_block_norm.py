"""The norms around a block and their gradients against 64-bit references, within bounds
that count roundings (``_block_ref``), and against differences."""

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _block_ref as B

pytestmark = pytest.mark.gpu

KIND = {"none": M.MEP_NORM_NONE, "rms": M.MEP_NORM_RMS, "layer": M.MEP_NORM_LAYER}
GATE = {"none": M.MEP_BLOCK_GATE_NONE, "token": M.MEP_BLOCK_GATE_TOKEN,
        "element": M.MEP_BLOCK_GATE_ELEMENT}
DTYPE = {"fp32": (M.MEP_FP32, torch.float32), "bf16": (M.MEP_BF16, torch.bfloat16)}
FILL = -7.0


class Case:
    """Inputs of one call on the GPU, and in 64 bits on the host."""

    def __init__(self, T, H, dtype, post="rms", pre="rms", gate="none", sigmoid=0, x=True, y=True,
                 weights=True, biases=False, a=1.0, c=1.0, offset=0.0, eps=1e-5, seed=0, mean=0.0):
        self.T, self.H, self.dtype, self.torch = T, H, dtype, DTYPE[dtype][1]
        self.post, self.pre, self.gate_kind, self.sigmoid = post, pre, gate, sigmoid
        self.cfg = M.MepNormConfig(H, DTYPE[dtype][0], KIND[post], KIND[pre], GATE[gate], sigmoid,
                                   eps, offset, a, c)
        f = lambda v: float(np.float32(v))  # noqa: E731  as the config holds it
        self.ref = dict(post=post, pre=pre, sigmoid=sigmoid, eps=f(eps), offset=f(offset), a=f(a),
                        c=f(c))
        rng = np.random.default_rng(seed)
        rows = lambda: mean + rng.standard_normal((T, H)) * (0.2 + 2 * rng.random((T, 1)))  # noqa: E731
        self.x = self.put(rows()) if x else None
        self.y = self.put(rows()) if y else None
        self.gate = None
        if gate == "token":
            self.gate = self.put(rng.standard_normal(T), torch.float32)
        elif gate == "element":
            self.gate = self.put(rng.standard_normal((T, H)))
        vec = lambda on, m: self.put(m + 0.3 * rng.standard_normal(H), torch.float32) if on else None  # noqa: E731
        self.wp, self.wn = vec(weights, 1.0), vec(weights, 1.0)
        self.bp, self.bn = vec(biases, 0.0), vec(biases, 0.0)
        self.gs, self.gn = self.put(rng.standard_normal((T, H))), self.put(rng.standard_normal((T, H)))

    def put(self, v, dtype=None):
        return torch.from_numpy(np.asarray(v, np.float32)).to(dtype or self.torch).cuda()

    def rows(self, dtype=None, cols=None):
        """An output with a row behind the last, which the call must leave."""
        return torch.full((self.T + 1, cols or self.H), FILL, device="cuda").to(dtype or self.torch)

    def forward(self, s=True, n=True, codes=False, stream=None):
        self.s, self.n = self.rows() if s else None, self.rows() if n else None
        self.codes = self.rows(torch.float8_e4m3fn) if codes else None
        self.scales = self.rows(torch.float32, self.H // 128) if codes else None
        M.mep_block_norm(self.cfg, self.x, self.y, self.gate, self.wp, self.bp, self.wn, self.bn,
                         self.T, self.s, self.n, self.codes, self.scales, stream)
        torch.cuda.synchronize()
        for t in (self.s, self.n, self.codes, self.scales):
            assert t is None or bool((t[self.T:].float() == FILL).all())

    def backward(self, stream_rows, want=None, stream=None):
        want = want or ("x", "y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")
        z = lambda n, t: torch.full_like(t, FILL) if n in want and t is not None else None  # noqa: E731
        col = lambda n, on: torch.full((self.H,), FILL, device="cuda") if n in want and on else None  # noqa: E731
        g = {"x": z("x", stream_rows), "y": z("y", self.y), "gate": z("gate", self.gate),
             "post_weight": col("post_weight", self.y is not None),
             "post_bias": col("post_bias", self.y is not None),
             "pre_weight": col("pre_weight", self.gn is not None),
             "pre_bias": col("pre_bias", self.gn is not None)}
        ws = torch.full((M.mep_block_norm_workspace_bytes(self.cfg, self.T),), 255,
                        dtype=torch.uint8, device="cuda")  # of any content
        M.mep_block_norm_backward(self.cfg, self.gs, self.gn, stream_rows, self.y, self.gate,
                                  self.wp, self.bp, self.wn, self.T, *g.values(), ws, stream)
        torch.cuda.synchronize()
        return {k: v for k, v in g.items() if v is not None}


def h64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, value, bound, what):
    got = h64(got) if torch.is_tensor(got) else got
    bad = ~(np.abs(got - value) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], value[bad][:3],
                           bound[bad][:3])


def check_forward(k, s=True, n=True, codes=False):
    k.forward(s, n, codes)
    (rs, es), (rn, en) = B.block_norm(k.ref, h64(k.x), h64(k.y), h64(k.gate), h64(k.wp), h64(k.bp),
                                      h64(k.wn), h64(k.bn))
    if s:
        close(k.s[:k.T], rs, B.rounded(rs, es, k.dtype), "s")
    if n:
        close(k.n[:k.T], rn, B.rounded(rn, en, k.dtype), "n")
    if codes:
        blocks = lambda v: v.reshape(k.T, -1, 128)  # noqa: E731
        scale = h64(k.scales)[:k.T]
        amax, most = np.abs(blocks(rn)).max(axis=2), blocks(en).max(axis=2)
        close(scale, amax / 448, (most + 2 * B.U32 * amax) / 448 + 1e-45, "scales")
        got = blocks(h64(k.codes)[:k.T]) * scale[:, :, None]
        # half a step of E4M3: 2^-4 of the value, at least 2^-10 of the scale
        close(got, blocks(rn), blocks(en) + np.maximum(2.0 ** -4 * np.abs(blocks(rn)), 2.0 ** -10
                                                       * scale[:, :, None]) * (1 + 2.0 ** -18),
              "codes")
    return k


SIZES = [(1, 8), (3, 64), (1, 7168), (257, 72), (70, 512), (33, 520), (40, 1024), (21, 1032),
         (5, 2048), (300, 2056), (9, 4104), (1100, 128), (17, 7168), (6, 8192), (5, 8200), (3, 16384)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "rms"),
                                      ("layer", "none")])
def test_forward(T, H, dtype, post, pre):
    gate = ("none", "token", "element")[(T + H // 8) % 3]
    check_forward(Case(T, H, dtype, post, pre, gate, sigmoid=T % 2, biases=post == "layer", a=0.5,
                       c=1.5, offset=1.0 if pre == "rms" else 0.0, seed=T + H))


# more rows than blocks, so that every block takes several, in each way of holding a row
MANY = [(3200, 72), (3200, 520), (1100, 1048), (1100, 2056), (520, 4104), (270, 8200)]


@pytest.mark.parametrize("T,H", MANY)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind,gate", [("rms", "token"), ("layer", "element")])
def test_many_rows(T, H, dtype, kind, gate):
    k = Case(T, H, dtype, kind, kind, gate, 1, biases=kind == "layer", seed=H)
    check_forward(k, codes=H % 128 == 0)
    check_backward(k)


# layer norms without biases or a gate for every element, and no gradients of biases, have
# kernels of their own
@pytest.mark.parametrize("T,H", SIZES + MANY)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "layer"), ("layer", "rms"),
                                      ("none", "layer"), ("layer", "none")])
def test_layer_norms_without_biases(T, H, dtype, post, pre):
    k = Case(T, H, dtype, post, pre, ("token", "none")[(T + H // 8) % 2], sigmoid=T % 2,
             weights=H % 3 != 0, a=0.5, c=1.5, offset=1.0 if pre == "rms" else 0.0, seed=T + H, mean=2.0)
    check_forward(k, codes=H % 128 == 0 and pre != "none")
    check_backward(k, ("x", "y", "gate", "post_weight", "pre_weight"))


@pytest.mark.parametrize("H", [264, 2056, 4104, 8200])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("without", ["gs", "gn", "y", "weights"])
def test_layer_norms_of_parts(H, dtype, without):
    k = Case(40, H, dtype, "layer", "layer", "none" if without == "y" else "token", 1,
             y=without != "y", weights=without != "weights", seed=H, mean=-1.0)
    check_forward(k)
    if without in ("gs", "gn"):
        setattr(k, without, None)
    whole, _, _ = check_backward(k, ("x", "y", "gate", "post_weight", "pre_weight"))
    some, _, _ = check_backward(k, ("y", "pre_weight"))
    assert all(torch.equal(t, whole[n]) for n, t in some.items())


@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("H", [1024, 1536])
def test_forward_gates(gate, sigmoid, H):
    check_forward(Case(37, H, "bf16", "rms", "rms", gate, sigmoid, seed=H))
    check_forward(Case(37, H, "fp32", "none", "rms", gate, sigmoid, weights=False, seed=H))


@pytest.mark.parametrize("T,H", [(1, 128), (30, 1024), (7, 1152), (129, 7168), (3, 16384)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_codes(T, H, dtype):
    k = check_forward(Case(T, H, dtype, "rms", "rms", "token", 1, seed=H), codes=True)
    if dtype == "fp32":  # the codes of exactly the rows that n holds
        n, scale = k.n[:T].cpu(), k.scales[:T].cpu()
        want = (n.reshape(T, -1, 128) * (1 / scale[:, :, None])).reshape(T, H).to(torch.float8_e4m3fn)
        assert torch.equal(want.view(torch.uint8), k.codes[:T].cpu().view(torch.uint8))
    check_forward(Case(T, H, dtype, "none", "rms", y=False, seed=H), s=False, n=False, codes=True)
    # without a norm the call only encodes rows
    check_forward(Case(T, H, dtype, "none", "none", y=False, weights=False, seed=H), s=False, n=False,
                  codes=True)


def test_codes_of_zero_tiny_and_non_finite_blocks():
    k = Case(6, 384, "fp32", "none", "none", y=False, weights=False)
    x = torch.randn((6, 384), generator=torch.Generator().manual_seed(2))
    x[0, :128] = 0.0
    x[1, 128:256] *= 1e-38 / 4     # scales below fp32's normal numbers
    x[2, 300] = float("inf")
    x[3, 7] = float("nan")
    x[4] *= 1e37
    x[5, 128:256] = float("nan")
    k.x = x.cuda()
    k.forward(True, True, True)
    codes, scale = k.codes[:6].cpu(), k.scales[:6].cpu()
    assert bool((codes[0, :128].float() == 0).all()) and float(scale[0, 0]) == 0
    value = codes.float().reshape(6, 3, 128) * scale[:, :, None]
    spoilt = torch.zeros((6, 3), dtype=torch.bool)
    spoilt[2, 2] = True               # an infinity spoils its block, a NaN only itself
    assert bool(torch.isnan(value[spoilt]).all())
    assert bool(torch.isnan(value[3, 0, 7])) and bool(torch.isnan(value[5, 1]).all())
    value[3, 0, 7], value[5, 1], x[3, 7], x[5, 128:256] = 0, 0, 0, 0
    assert bool(torch.isfinite(value[~spoilt]).all())
    off = (value - x.reshape(6, 3, 128)).abs()
    lim = torch.maximum(x.reshape(6, 3, 128).abs() / 16, scale[:, :, None] / 1024) * 1.001
    lim[1, 1] = scale[1, 1] * 32   # the scale itself has few bits there: its half-step times 448
    assert bool((off <= lim)[~spoilt].all())


@pytest.mark.parametrize("H", [256, 4096])
@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_zero_constant_and_large_rows(pre, H):
    k = Case(4, H, "fp32", "none", pre, y=False, seed=3)
    k.x[0] = 0.0
    k.x[1] = 3.0
    k.x[2] *= 1e15
    k.x[3] *= 1e-20
    check_forward(k)


def test_parts_that_are_not_there():
    check_forward(Case(9, 640, "bf16", x=False, seed=1))           # no residual
    check_forward(Case(9, 640, "bf16", y=False, seed=1))           # no block
    check_forward(Case(9, 640, "bf16", seed=1), n=False)           # the stream alone
    check_forward(Case(9, 640, "bf16", seed=1), s=False)
    check_forward(Case(9, 640, "bf16", weights=False, biases=True, seed=1))
    k = Case(0, 640, "bf16")
    k.forward()                                                    # no rows


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H", [640, 2056])
def test_in_place(dtype, H):
    k = Case(300, H, dtype, "rms", "layer", "token", 1, seed=4)
    k.forward()
    s, n = k.s[:300].clone(), k.n[:300].clone()
    x, y = k.x.clone(), k.y.clone()
    M.mep_block_norm(k.cfg, x, y, k.gate, k.wp, k.bp, k.wn, k.bn, 300, x, y, None, None)
    torch.cuda.synchronize()
    assert torch.equal(x, s) and torch.equal(y, n)
    want = k.backward(k.x)
    gs, y = k.gs.clone(), k.y.clone()
    ws = torch.zeros(M.mep_block_norm_workspace_bytes(k.cfg, 300), dtype=torch.uint8, device="cuda")
    M.mep_block_norm_backward(k.cfg, gs, k.gn, k.x, y, k.gate, k.wp, k.bp, k.wn, 300, gs, y, None,
                              None, None, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(gs, want["x"]) and torch.equal(y, want["y"])


# ---- gradients ---------------------------------------------------------------

def reference_gradients(k, s):
    return B.block_norm_backward(k.ref, h64(k.gs), h64(k.gn), h64(s), h64(k.y), h64(k.gate),
                                 h64(k.wp), h64(k.bp), h64(k.wn), max(1, k.T))


def check_backward(k, want=None):
    s = k.x if k.x is not None else k.put(np.random.default_rng(8).standard_normal((k.T, k.H)))
    got = k.backward(s, want)
    ref = reference_gradients(k, s)
    assert want is None or set(want) >= set(got)
    for name, t in got.items():
        value, err = ref[name]
        vector = name.startswith(("p", "b")) or (name == "gate" and k.gate_kind == "token")
        close(t, value, B.rounded(value, err, "fp32" if vector else k.dtype), name)
    return got, ref, s


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "rms"),
                                      ("layer", "none")])
def test_backward(T, H, dtype, post, pre):
    gate = ("token", "element", "none")[(T + H // 8) % 3]
    check_backward(Case(T, H, dtype, post, pre, gate, sigmoid=T % 2, biases=post == "layer", a=0.5,
                        c=1.5, offset=1.0 if pre == "rms" else 0.0, seed=T + H))


@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("H", [1024, 1536])
def test_backward_gates(gate, sigmoid, H):
    check_backward(Case(600, H, "bf16", "rms", "rms", gate, sigmoid, seed=H))
    check_backward(Case(37, H, "fp32", "none", "rms", gate, sigmoid, weights=False, biases=True, seed=H))


def test_backward_of_what_is_asked():
    full, _, _ = check_backward(Case(50, 640, "bf16", "rms", "layer", "token", 1, biases=True, seed=2))
    for want in (("x",), ("y",), ("gate",), ("post_weight",), ("pre_bias",), ("post_bias", "pre_weight"),
                 ("x", "pre_weight")):
        k = Case(50, 640, "bf16", "rms", "layer", "token", 1, biases=True, seed=2)
        got, _, _ = check_backward(k, want)
        assert set(got) == set(want)
        assert all(torch.equal(got[n], full[n]) for n in want)
    k = Case(50, 640, "bf16", seed=2)
    k.gs = None
    check_backward(k)                            # of n alone
    k = Case(50, 640, "bf16", "layer", seed=2)
    k.gn = None
    check_backward(k)                            # of s alone
    k = Case(50, 640, "bf16", y=False, seed=2)
    check_backward(k)                            # no block
    k = Case(0, 640, "bf16", seed=2)
    got = k.backward(k.x)
    assert all(bool((got[n] == 0).all()) for n in ("post_weight", "post_bias", "pre_weight", "pre_bias"))


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms"), ("none", "none")])
@pytest.mark.parametrize("gate", ["token", "element"])
def test_gradients_are_the_definitions(post, pre, gate):
    """By differentiating the forward formula in 64 bits, and by its differences along a
    random direction of all inputs at once."""
    k = Case(24, 264, "fp32", post, pre, gate, 1, biases=True, a=0.7, c=1.3, offset=1.0, seed=11)
    names = ("x", "y", "gate", "wp", "bp", "wn", "bn")
    inputs = {n: getattr(k, n).cpu().double().requires_grad_(True) for n in names}
    gs, gn = k.gs.cpu().double(), k.gn.cpu().double()

    def hat(kind, u):
        if kind == "layer":
            u = u - u.mean(1, keepdim=True)
        return u if kind == "none" else u / torch.sqrt((u * u).mean(1, keepdim=True) + k.ref["eps"])

    def total(i):
        g = torch.sigmoid(i["gate"])
        v = hat(post, i["y"]) * (1 + i["wp"]) + i["bp"]
        s = k.ref["a"] * i["x"] + k.ref["c"] * (g[:, None] if gate == "token" else g) * v
        n = hat(pre, s) * (1 + i["wn"]) + i["bn"]
        return (s * gs).sum() + (n * gn).sum(), s

    loss, s = total(inputs)
    want = dict(zip(names, torch.autograd.grad(loss, list(inputs.values()))))
    stream = s.detach().float().cuda()
    got = k.backward(stream)
    ref = reference_gradients(k, stream)
    called = dict(zip(names, ("x", "y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")))
    # the stream rounds to fp32 on its way: a half-step of every value, through a norm
    # whose second derivative is below 8 r^2 |g| at these rows: far below 1e-5 of the norm
    for n in names:
        off = (got[called[n]].cpu().double() - want[n]).norm() / want[n].norm()
        assert off <= 1e-5, (n, off)
        value = torch.from_numpy(ref[called[n]][0])
        assert (value - want[n]).norm() <= 1e-5 * want[n].norm(), n
    rng = torch.Generator().manual_seed(1)
    d = {n: torch.randn(t.shape, generator=rng, dtype=torch.float64) for n, t in inputs.items()}
    h = 1e-6
    with torch.no_grad():
        up, _ = total({n: inputs[n] + h * d[n] for n in names})
        down, _ = total({n: inputs[n] - h * d[n] for n in names})
    slope = sum(float((got[called[n]].cpu().double() * d[n]).sum()) for n in names)
    size = sum(float((want[n] * d[n]).norm()) for n in names)
    # fp32 gradients 1e-5 of their norms at most, differences h^2 and 1e-16/h of the sums
    assert abs(float(up - down) / (2 * h) - slope) <= 1e-5 * size + 1e-8 * float(gn.abs().sum())


@pytest.mark.parametrize("H", [2056, 4104, 8200])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_threads_past_the_row_hold_no_weights(kind, H):
    # NaN weights of a longer row before it: what they leave in LDS reaches no sum
    left = Case(300, 16384 if H > 8192 else 8192, "bf16", kind, kind, biases=True, seed=1)
    for w in (left.wp, left.wn, left.bp):
        w.fill_(float("nan"))
    for _ in range(3):
        left.backward(left.x)
        check_backward(Case(300, H, "bf16", kind, kind, "token", 1, seed=H))


def test_results_repeat():
    k = Case(2000, 1536, "bf16", "rms", "rms", "token", 1, seed=5)
    a, b = k.backward(k.x), k.backward(k.x)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_long_batch():
    # rows past 2^31 elements
    T, H = (1 << 31) // 16384 + 3, 16384
    cfg = M.MepNormConfig(H, M.MEP_BF16, M.MEP_NORM_NONE, M.MEP_NORM_RMS, 0, 0, 1e-6, 0.0, 1.0, 1.0)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, H), generator=torch.Generator().manual_seed(3)).cuda()
    n = torch.zeros_like(x)
    M.mep_block_norm(cfg, x, None, None, None, None, None, None, T, None, n, None, None)
    torch.cuda.synchronize()
    small = torch.zeros((3, H), dtype=torch.bfloat16, device="cuda")
    M.mep_block_norm(cfg, x[-3:].contiguous(), None, None, None, None, None, None, 3, None, small, None,
                     None)
    assert torch.equal(n[-3:], small) and bool(small.any()) and not bool(n[:-3].any())


# a layer's config serves its first rows too, which no block stands before: the gate that
# it names is not there then.  More rows than blocks in the last size of each width.
@pytest.mark.parametrize("T,H", [(1, 128), (3, 640), (3200, 640), (1100, 2048), (600, 7168), (5, 8320),
                                 (300, 16384)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", ["token", "element"])
@pytest.mark.parametrize("sigmoid", [0, 1])
def test_config_with_a_gate_and_no_block(T, H, dtype, gate, sigmoid):
    k = Case(T, H, dtype, "rms", "rms", "none", sigmoid, y=False, seed=H)
    want = []
    for outs in ((True, True, True), (False, True, False), (False, False, True)):
        k.cfg.gate = GATE["none"]
        k.forward(*outs)
        want.append((k.s, k.n, k.codes, k.scales))
    k.cfg.gate = GATE[gate]
    for outs, w in zip(((True, True, True), (False, True, False), (False, False, True)), want):
        k.forward(*outs)
        for a, b in zip((k.s, k.n, k.codes, k.scales), w):
            assert (a is None) == (b is None)
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check_forward(k, codes=True)
    check_backward(k, ("x", "pre_weight", "pre_bias"))


def test_codes_of_blocks_whose_scales_have_few_bits():
    # a block's largest value by steps of fp32's smallest number, the others random below
    # it: every finite block has finite codes, whatever amax / 448 rounds to
    amax = np.r_[np.arange(1, 8192), 2 ** np.arange(13, 24), 3 * 2 ** np.arange(12, 22) + 1]
    H = 128 * 64
    amax = np.resize(amax, (len(amax) + 63) // 64 * 64)
    rng = np.random.default_rng(6)
    steps = np.round(rng.uniform(-1, 1, (len(amax), 128)) * amax[:, None])
    steps[np.arange(len(amax)), rng.integers(0, 128, len(amax))] = amax * rng.choice([-1, 1], len(amax))
    k = Case(len(amax) // 64, H, "fp32", "none", "none", y=False, weights=False)
    k.x = torch.from_numpy((steps * 2.0 ** -149).astype(np.float32).reshape(k.T, H)).cuda()
    k.forward(False, False, True)
    scale = h64(k.scales)[:k.T].reshape(-1, 1) * 2.0 ** 149
    got = h64(k.codes)[:k.T].reshape(-1, 128)
    assert np.isfinite(got).all()
    assert np.array_equal(scale[:, 0], np.round(amax / 448.0))  # to the nearest, even, step
    # half a step of the code, or what the largest code does not reach: 448 times the half
    # step that the scale may lie below amax / 448
    off = np.abs(got * scale - steps)
    lim = np.maximum(np.abs(steps) / 16, scale / 1024) * (1 + 2.0 ** -18)
    past = np.abs(steps) > 448 * scale
    assert bool((off <= np.where(past, 224.0, lim)).all())
    assert bool((np.abs(got[past & (scale > 0)]) == 448).all()) and past.any()


@pytest.mark.parametrize("H", [256, 4096, 16384])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_whose_squares_just_fit(kind, H):
    # equal magnitudes, the row's sum of squares 0.95 of fp32's largest number (the gradients
    # 1e-3 of it, whose products with the rows are sums as well)
    size = np.sqrt(0.95 * float(np.finfo(np.float32).max) / H)
    sign = np.random.default_rng(H).choice([-1.0, 1.0], (5, H))
    sign[:, ::2] = -sign[:, 1::2]     # their mean is 0, so that a layer norm takes off nothing
    k = Case(5, H, "fp32", "none", kind, y=False, seed=H)
    k.x = k.put(size * sign)
    check_forward(k, codes=True)
    k.x = k.put(1e-3 * size * sign)
    check_backward(k)
    k = Case(5, H, "fp32", kind, "none", x=False, seed=H)
    k.y = k.put(size * sign)
    check_forward(k)


@pytest.mark.parametrize("H", [72, 520, 2056, 4104, 8200])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind,biases", [("rms", False), ("layer", False), ("layer", True)])
def test_gradients_of_the_stream_alone_pass_by_the_next_norm(H, dtype, kind, biases):
    # without grad_n the next norm hands nothing back, whatever its weights are
    k = Case(9, H, dtype, kind, kind, "token", 1, biases=biases, seed=H)
    k.gn = None
    want = ("x", "y", "gate", "post_weight")
    whole, _, _ = check_backward(k, want)
    k.wn[3], k.wn[4] = float("inf"), float("nan")
    got = k.backward(k.x, want)
    assert all(torch.equal(got[n], whole[n]) for n in want)
    got = k.backward(k.x, ("x",))
    assert torch.equal(got["x"], whole["x"])


# codes and scales of rows that a block takes after its first, in each way of holding a row
# and each kind of kernel
@pytest.mark.parametrize("T,H", [(3200, 128), (3200, 640), (1100, 1152), (1100, 2048), (600, 7168),
                                 (300, 8320)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind,gate,biases", [("rms", "token", False), ("layer", "token", False),
                                              ("layer", "element", True)])
def test_codes_of_many_rows(T, H, dtype, kind, gate, biases):
    k = Case(T, H, dtype, kind, kind, gate, 1, biases=biases, seed=H)
    check_forward(k, codes=True)
    # a row's codes do not depend on which block took it, nor on the rows around it
    codes, scales = k.codes[:T].view(torch.uint8).clone(), k.scales[:T].clone()
    at = torch.randperm(T, generator=torch.Generator().manual_seed(T)).cuda()
    k.x, k.y, k.gate = k.x[at].contiguous(), k.y[at].contiguous(), k.gate[at].contiguous()
    k.forward(False, False, True)
    assert torch.equal(k.codes[:T].view(torch.uint8), codes[at]) and torch.equal(k.scales[:T], scales[at])


@pytest.mark.parametrize("T,H", [(1, 128), (9, 256), (5, 1536), (3, 7168), (2, 16384)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate,biases", [("element", False), ("none", True), ("element", True)])
def test_codes_with_biases_or_a_gate_for_every_element(T, H, dtype, gate, biases):
    check_forward(Case(T, H, dtype, "rms", "rms", gate, 1, biases=biases, offset=1.0, seed=H), codes=True)


@pytest.mark.parametrize("T,H", [(3200, 72), (4096, 512), (3200, 1024), (1100, 1048), (1100, 2056),
                                 (520, 4104), (600, 7168), (270, 8200)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind,gate,biases", [("rms", "token", False), ("layer", "token", False),
                                              ("layer", "element", True)])
def test_column_sums_within_their_depth(T, H, dtype, kind, gate, biases):
    # A thread adds up one row in `blocks` (of 4 rows each up to 1024 columns), the waves of
    # such a block are joined by 3 additions, and the rest is added in fp64 and rounded once:
    # so many roundings of the magnitudes added are allowed, not one for every row.
    k = Case(T, H, dtype, kind, kind, gate, 1, biases=biases, seed=H)
    blocks = min(256, M.mep_block_norm_workspace_bytes(k.cfg, T) // (16 * H))
    depth = -(-T // (blocks * (4 if H <= 1024 else 1)))
    assert depth <= 16
    want = ("post_weight", "pre_weight") + (("post_bias", "pre_bias") if biases else ())
    got = k.backward(k.x, want)
    ref = B.block_norm_backward(k.ref, h64(k.gs), h64(k.gn), h64(k.x), h64(k.y), h64(k.gate), h64(k.wp),
                                h64(k.bp), h64(k.wn), depth + 3)
    assert set(got) == set(want)
    for name, t in got.items():
        close(t, ref[name][0], B.rounded(*ref[name], "fp32"), name)


@pytest.mark.parametrize("T,H", [(3200, 640), (1100, 1152), (1100, 2056), (600, 7168), (300, 8200)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind,gate", [("rms", "token"), ("layer", "element")])
def test_in_place_of_many_rows(T, H, dtype, kind, gate):
    # the loads of a block's next rows run ahead of the stores over its present one
    k = Case(T, H, dtype, kind, kind, gate, 1, biases=gate == "element", seed=H)
    k.forward()
    s, n = k.s[:T].clone(), k.n[:T].clone()
    call = lambda x, y, s, n: M.mep_block_norm(k.cfg, x, y, k.gate, k.wp, k.bp, k.wn, k.bn, T, s, n,  # noqa: E731
                                               None, None)
    for s_of, n_of in (("x", "y"), ("y", None), (None, "y"), ("x", None)):
        rows = {"x": k.x.clone(), "y": k.y.clone(), None: torch.zeros_like(k.x)}
        out_s, out_n = rows[s_of], rows[n_of]
        if s_of is None or n_of is None:
            other = torch.zeros_like(k.x)
            out_s, out_n = (other, out_n) if s_of is None else (out_s, other)
        call(rows["x"], rows["y"], out_s, out_n)
        assert torch.equal(out_s, s) and torch.equal(out_n, n), (s_of, n_of)
    want = k.backward(k.x)
    gs, y = k.gs.clone(), k.y.clone()
    ws = torch.zeros(M.mep_block_norm_workspace_bytes(k.cfg, T), dtype=torch.uint8, device="cuda")
    cols = [torch.zeros(H, device="cuda") for _ in range(4)]
    cols = [c if gate == "element" or i % 2 == 0 else None for i, c in enumerate(cols)]
    of_gate = torch.zeros_like(k.gate)
    M.mep_block_norm_backward(k.cfg, gs, k.gn, k.x, y, k.gate, k.wp, k.bp, k.wn, T, gs, y, of_gate, *cols, ws)
    torch.cuda.synchronize()
    if gate == "element":
        assert torch.equal(gs, want["x"]) and torch.equal(y, want["y"]) and torch.equal(of_gate, want["gate"])
    apart = k.backward(k.x, ("x", "y", "gate", "post_weight", "pre_weight") +
                       (("post_bias", "pre_bias") if gate == "element" else ()))
    got = dict(zip(("post_weight", "post_bias", "pre_weight", "pre_bias"), cols), x=gs, y=y, gate=of_gate)
    assert all(torch.equal(got[n], apart[n]) for n in apart)


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1e-38])
@pytest.mark.parametrize("H", [72, 7168])
def test_zero_rows_and_the_smallest_eps(eps, H):
    k = Case(4, H, "fp32", "rms", "rms", x=False, eps=eps, seed=H)
    k.y[1], k.y[2] = 0.0, 1e-12
    check_forward(k)
    assert not bool(k.n[1].any()) and not bool(k.s[1].any())


def test_codes_on_both_sides_of_the_lifted_scales():
    # scales from 2^-130 to 2^-122, and NaN among values that are held to 448 scales
    H = 128 * 8
    x = torch.randn((64, H), generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    amax = x.reshape(64, 8, 128).abs().amax(2)
    e = 448 * 2.0 ** (-130 + 8 * torch.arange(512, dtype=torch.float64).reshape(64, 8) / 511)
    x = (x.reshape(64, 8, 128) * (e / amax)[:, :, None]).float().reshape(64, H)
    x[7, 130] = float("nan")
    k = Case(64, H, "fp32", "none", "none", y=False, weights=False)
    k.x = x.cuda()
    k.forward(False, False, True)
    scale, got = h64(k.scales)[:64, :, None], h64(k.codes)[:64].reshape(64, 8, 128)
    v = x.double().numpy().reshape(64, 8, 128)
    assert np.isnan(got[7, 1, 2]) and np.isnan(got).sum() == 1
    got[7, 1, 2] = v[7, 1, 2] = 0.0
    # the scale is within half a step of fp32, which is 2^-150 at least; so is the largest
    # value beyond 448 scales at most 448 times that
    assert bool((np.abs(scale[..., 0] - np.abs(v).max(2) / 448) <= scale[..., 0] * B.U32 + 2.0 ** -150).all())
    lim = np.maximum(np.abs(v) / 16, scale / 1024) * (1 + 2.0 ** -18)
    assert bool((np.abs(got * scale - v) <= lim).all())
