"""The norm of many gradients and their clipping against 64-bit references."""

import math

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _experts_ref as R

pytestmark = pytest.mark.gpu


def make(sizes, scale=1.0, seed=0, dtypes=(torch.bfloat16, torch.float32)):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dtypes[i % len(dtypes)]).cuda()
            for i, n in enumerate(sizes)]


def norm_of(lst, stream=None):
    ws = torch.zeros(M.mep_grad_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
    norm = torch.full((4,), -7.0, device="cuda")
    M.mep_grad_norm(lst, norm, ws, stream)
    torch.cuda.synchronize()
    assert bool((norm[1:] == -7).all())
    return norm, ws


def exact(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def check_norm(got, want):
    # summed in fp64 and rounded once
    assert abs(float(got) - want) <= 1.01 * R.U32 * want, (float(got), want)


SIZES = [[1], [7], [8], [0], [], [16384], [16385], [8191, 8193, 3], [0, 5, 0, 0, 70001, 0],
         [1 << 20, 1, 33333], [5] * 127, [17 + i for i in range(128)], [9] * 129, [100 + i for i in range(700)]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0] if s else 0}")
def test_norm_and_clip(sizes):
    grads = make(sizes)
    lst = M.MepGrads(grads)
    norm, _ = norm_of(lst)
    want = exact(grads)
    check_norm(norm[0], want)
    for limit in (0.3, 1e9) if want else (1.0,):
        outs = [torch.full((t.numel() + 9,), -7.0, device="cuda").to(t.dtype) for t in grads]
        M.mep_grad_clip(M.MepGrads(grads, [o[:t.numel()] for o, t in zip(outs, grads)]), norm, limit)
        torch.cuda.synchronize()
        f = min(1.0, limit / (float(norm[0]) + 1e-6))
        for t, o in zip(grads, outs):
            n = t.numel()
            assert bool((o[n:] == -7).all())
            ref = f * t.double()
            u = R.UBF16 if t.dtype == torch.bfloat16 else R.U32
            # the factor within 2 half-steps of fp32 (sum and quotient), the product's rounding
            assert bool(((o[:n].double() - ref).abs() <= (u + 3 * R.U32) * ref.abs() + 1e-45).all())
            if f == 1.0:
                assert torch.equal(o[:n], t)


def test_in_place():
    grads = make([1000, 70000, 13], scale=3.0)
    before = [t.clone() for t in grads]
    lst = M.MepGrads(grads)
    norm, _ = norm_of(lst)
    M.mep_grad_clip(lst, norm, 1e9)         # below the limit: as they were
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    outs = [torch.zeros_like(t) for t in grads]
    M.mep_grad_clip(M.MepGrads(grads, outs), norm, 1.0)
    M.mep_grad_clip(lst, norm, 1.0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    again, _ = norm_of(lst)
    # every value within half a step of bf16 of its exact multiple: so is the norm
    assert abs(float(again[0]) - 1.0) <= R.UBF16 + 1e-5


def test_norms_of_ranks_joined():
    # each rank's own norm, put together on the device, clips as one list would
    a, b = make([5000, 31], seed=1), make([777], seed=2)
    na, _ = norm_of(M.MepGrads(a))
    nb, _ = norm_of(M.MepGrads(b))
    both = torch.sqrt(na[:1].double() ** 2 + nb[:1].double() ** 2).float()
    # two roundings in turn: each rank's norm within half a step, so their root of squares
    # (whose relative error is a mean of theirs), and the rounding of that
    want = exact(a + b)
    assert abs(float(both[0]) - want) <= 2.01 * R.U32 * want
    M.mep_grad_clip(M.MepGrads(a + b), both, 1.0)
    torch.cuda.synchronize()
    assert abs(exact(a + b) - 1.0) <= R.UBF16 + 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-30, 1e-38, 1e25, 3e38])
def test_squares_neither_vanish_nor_overflow(scale, dtype):
    t = (torch.rand(5000, generator=torch.Generator().manual_seed(1)) * scale).to(dtype).cuda()
    norm, _ = norm_of(M.MepGrads([t]))
    want = exact([t])
    if want > 3.4e38:
        assert math.isinf(float(norm[0]))
    elif want > 1.2e-38:
        check_norm(norm[0], want)
    else:
        assert abs(float(norm[0]) - want) <= 1e-45


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite(bad):
    grads = make([100, 40000], dtypes=(torch.float32, torch.bfloat16))
    grads[1][39999] = bad
    norm, ws = norm_of(M.MepGrads(grads))
    got = float(norm[0])
    assert math.isnan(got) if math.isnan(bad) else got == math.inf
    outs = [torch.ones_like(t) for t in grads]
    M.mep_grad_clip(M.MepGrads(grads, outs), norm, 1.0)
    torch.cuda.synchronize()
    if math.isnan(bad):
        assert all(bool(torch.isnan(o).all()) for o in outs)
    else:
        assert bool((outs[0] == 0).all()) and bool((outs[1][:-1] == 0).all())
        assert math.isnan(float(outs[1][-1]))
    # the workspace is ready for the next call all the same
    grads[1][39999] = 1.0
    M.mep_grad_norm(M.MepGrads(grads), norm, ws)
    torch.cuda.synchronize()
    check_norm(norm[0], exact(grads))


def test_tensor_past_2_31_elements():
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-5:] = 3.0
    t[5] = 4.0
    lst = M.MepGrads([t])
    norm, _ = norm_of(lst)
    check_norm(norm[0], math.sqrt(16 + 45))
    M.mep_grad_clip(lst, norm, 1.0)
    torch.cuda.synchronize()
    f = 1.0 / (math.sqrt(61) + 1e-6)
    assert bool(((t[-5:].double() - 3 * f).abs() <= (R.UBF16 + 3 * R.U32) * 3 * f).all())
    assert abs(float(t[5]) - 4 * f) <= (R.UBF16 + 3 * R.U32) * 4 * f
    assert int((t != 0).sum()) == 6


def test_workspace_is_used_again_and_results_repeat():
    grads = make([123457, 1000, 65536 * 3 + 1])
    lst = M.MepGrads(grads)
    norm, ws = norm_of(lst)
    first = float(norm[0])
    for _ in range(20):
        M.mep_grad_norm(lst, norm, ws)
    torch.cuda.synchronize()
    assert float(norm[0]) == first


def test_graph_replays():
    grads = make([70001, 300] + [50 + i for i in range(200)])
    outs = [torch.zeros_like(t) for t in grads]
    lst = M.MepGrads(grads, outs)
    norm, ws = norm_of(lst)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mep_grad_norm(lst, norm, ws)
        M.mep_grad_clip(lst, norm, 2.0)
    for seed in (3, 1, 4, 1):
        new = make([t.numel() for t in grads], seed=seed)
        for t, v in zip(grads, new):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        check_norm(norm[0], exact(new))
        got, n = [o.clone() for o in outs], float(norm[0])
        M.mep_grad_norm(lst, norm, ws)      # eagerly, between replays, on the same workspace
        M.mep_grad_clip(lst, norm, 2.0)
        torch.cuda.synchronize()
        assert float(norm[0]) == n and all(torch.equal(a, b) for a, b in zip(got, outs))


def test_lists_on_two_streams_at_once():
    lists = [make([300000 + i, 77], seed=i) for i in range(2)]
    wants = [exact(g) for g in lists]
    objs = [M.MepGrads(g) for g in lists]
    spaces = [torch.zeros(M.mep_grad_workspace_bytes(o), dtype=torch.uint8, device="cuda") for o in objs]
    norms = [torch.zeros(1, device="cuda") for _ in objs]
    streams = [torch.cuda.Stream() for _ in objs]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, s, n, w in zip(objs, streams, norms, spaces):
            with torch.cuda.stream(s):
                M.mep_grad_norm(o, n, w)
    torch.cuda.synchronize()
    for n, w in zip(norms, wants):
        check_norm(n[0], w)


def test_lists_that_are_refused():
    a, b = make([8, 8])
    with pytest.raises(ValueError, match="same type"):
        M.MepGrads([a], [b])
    with pytest.raises(ValueError, match="fp32 or bf16"):
        M.MepGrads([a.half()])
    with pytest.raises(ValueError, match="values"):
        M.MepGrads([a], [a[:4]])
    with pytest.raises(ValueError, match="outs for"):
        M.MepGrads([a, b], [a])
    with pytest.raises(ValueError, match="contiguous"):
        M.MepGrads([torch.zeros((4, 4), device="cuda").t()[:2]])
    with pytest.raises(ValueError, match="on the GPU"):
        M.MepGrads([torch.zeros(4)])
    flat = torch.zeros(64, device="cuda")
    for grads in ([a, a], [flat[:32], flat[16:48]]):
        with pytest.raises(ValueError, match="overlap"):
            M.MepGrads(grads)
    with pytest.raises(ValueError, match="overlap"):
        M.MepGrads([flat[:16], flat[32:48]], [flat[48:], flat[:16]])   # an out over another's gradient
    with pytest.raises(ValueError, match="overlap"):
        M.MepGrads([flat[:16]], [flat[8:24]])                          # over its own, moved
    M.MepGrads([flat[:16], flat[:16], flat[8:40]], [torch.zeros_like(t) for t in
                                                    (flat[:16], flat[:16], flat[8:40])])
    M.MepGrads([flat[:16], flat[16:32], flat[:0]])                     # neighbours are no overlap
    lst = M.MepGrads([a])
    norm, ws = norm_of(lst)
    with pytest.raises(M.MepError) as e:
        M.mep_grad_norm(lst, norm, ws[:-1])
    assert e.value.code == M.MEP_ERR_SHAPE
    with pytest.raises(M.MepError) as e:
        M.mep_grad_clip(M.MepGrads([a[1:5]]), norm, 1.0)
    assert e.value.code == M.MEP_ERR_ALIGN
    with pytest.raises(ValueError, match="norm"):
        M.mep_grad_norm(lst, norm.double(), ws)


@pytest.mark.parametrize("worst", [1.0, math.inf, -math.inf, math.nan])
def test_no_limit(worst):
    # an infinite limit: gradients stay as they are, infinite ones too, unless the norm is NaN
    grads = make([100, 40000, 7], dtypes=(torch.float32, torch.bfloat16))
    grads[1][123] = worst
    norm, _ = norm_of(M.MepGrads(grads))
    outs = [torch.zeros_like(t) for t in grads]
    M.mep_grad_clip(M.MepGrads(grads, outs), norm, math.inf)
    own = [t.clone() for t in grads]
    M.mep_grad_clip(M.MepGrads(own), norm, math.inf)
    torch.cuda.synchronize()
    for g, o, i in zip(grads, outs, own):
        if math.isnan(worst):
            assert bool(torch.isnan(o).all()) and bool(torch.isnan(i).all())
        else:
            assert torch.equal(o, g) and torch.equal(i, g)
