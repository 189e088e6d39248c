"""The router over groups of experts against 64-bit references: every size of row, groups of
one expert and one group of all, ties, scores closer than fp32 tells, masks and NaN."""

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _block_ref as B
import _experts_ref as R

pytestmark = pytest.mark.gpu

SCORE = {"softmax": M.MEP_SCORE_SOFTMAX, "sigmoid": M.MEP_SCORE_SIGMOID}
BY = {"max": M.MEP_GROUP_MAX, "top2": M.MEP_GROUP_TOP2}
DTYPE = {"fp32": (M.MEP_FP32, torch.float32), "bf16": (M.MEP_BF16, torch.bfloat16)}


def run(x, bias, k, score, normalize, scale, G, top, by, dtype, stream=None):
    """x: host fp32; (indices, weights, the logits as the type holds them)."""
    T, E = x.shape
    cfg = M.MepGateConfig(E, k, SCORE[score], DTYPE[dtype][0], normalize, scale, 0.0)
    logits = torch.from_numpy(x).to(DTYPE[dtype][1]).cuda()
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    M.mep_gate_grouped(cfg, G, top, BY[by], logits, b, T, idx, w, stream)
    torch.cuda.synchronize()
    assert bool((idx[T:] == -7).all()) and bool((w[T:] == -7).all())  # nothing behind the last row
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy(), logits.double().cpu().numpy()


def check(x, bias, k, score, G, top, by, dtype, normalize=1, scale=1.0, weights=True):
    idx, w, x64 = run(x, bias, k, score, normalize, scale, G, top, by, dtype)
    ridx, rw = B.grouped(x64, bias, k, score, normalize, scale, G, top, by)
    bad = np.argwhere(idx != ridx)
    assert not len(bad), (len(bad), bad[:3], idx[bad[0][0]], ridx[bad[0][0]])
    if weights:
        assert np.all(np.abs(w - rw) <= R.prob_steps() * R.U32 * np.abs(rw))


# (T, E, groups, top groups, k): rows of every layout, a group inside a lane's values and
# over several lanes, groups of odd sizes, of one expert, and all experts in one
SIZES = [(1, 256, 8, 4, 8), (1, 1, 1, 1, 1), (3, 8, 8, 3, 3), (5, 33, 3, 1, 11), (257, 60, 6, 2, 4),
         (64, 64, 4, 2, 6), (130, 66, 11, 5, 7), (77, 128, 16, 3, 3), (100, 128, 64, 9, 9),
         (300, 256, 8, 4, 8), (65, 256, 2, 1, 10), (41, 256, 64, 60, 8), (33, 300, 10, 9, 17),
         (40, 512, 16, 1, 10), (21, 512, 4, 3, 5), (19, 513, 27, 5, 8), (9, 1000, 8, 2, 32),
         (7, 1024, 32, 4, 5), (7, 1608, 8, 7, 12), (5, 4096, 64, 8, 32), (70, 256, 1, 1, 8)]


@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,G,top,k", SIZES)
def test_sizes(T, E, G, top, k, dtype, by, score, bias):
    if by == "top2" and E == G:
        pytest.skip("two experts a group at least")
    rng = np.random.default_rng(T * 1000 + E)
    x = np.clip(rng.standard_normal((T, E)) * 2, -12, 12).astype(np.float32)
    b = (rng.standard_normal(E) * 0.2).astype(np.float32) if bias else None
    check(x, b, k, score, G, top, by, dtype, T % 2, 2.5)


def test_all_groups_give_the_plain_router():
    rng = np.random.default_rng(3)
    T, E, k = 300, 120, 6
    x = rng.standard_normal((T, E)).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    idx, w, _ = run(x, b, k, "sigmoid", 1, 1.5, 6, 6, "top2", "bf16")
    cfg = M.MepGateConfig(E, k, M.MEP_SCORE_SIGMOID, M.MEP_BF16, 1, 1.5, 0.0)
    pi = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    pw = torch.zeros((T, k), device="cuda")
    M.mep_gate(cfg, torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(b).cuda(), T, pi, pw)
    assert np.array_equal(idx, pi.cpu().numpy()) and np.array_equal(w, pw.cpu().numpy())


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("score,bias", [("softmax", None), ("sigmoid", None), ("sigmoid", "zero"),
                                        ("sigmoid", "two values")])
def test_ties_go_to_the_lowest(score, bias, by):
    # logits of four values only: groups and experts are chosen among equals
    T, E, k = 200, 96, 8
    rng = np.random.default_rng(3)
    x = rng.choice([-1.5, 0.0, -0.0, 2.0], size=(T, E)).astype(np.float32)
    b = None if bias is None else np.zeros(E, np.float32)
    if bias == "two values":
        b[::3] = 0.125
    for G, top in ((8, 3), (32, 5), (3, 1)):
        check(x, b, k, score, G, top, by, "bf16")
    check(np.zeros((3, E), np.float32), b, k, score, 8, 4, by, "fp32")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_closer_than_fp32_tells(score):
    # the two best of every group sum to nearly the same: one group's are a fp32 step of
    # the logits apart from another's, which leaves the sums equal in fp32
    T, G, S, k = 128, 8, 16, 8
    rng = np.random.default_rng(7)
    x = np.full((T, G, S), -8.0, np.float32)
    step = np.stack([rng.permutation(G) for _ in range(T)]).astype(np.float32)
    x[:, :, 3] = np.float32(3.0) + step * np.float32(2 ** -22)
    x[:, :, 9] = np.float32(2.5)
    b = np.ones(G * S, np.float32) if score == "sigmoid" else None
    if score == "sigmoid":
        s32 = (1 / (1 + np.exp(-x[:, :, 3]))).astype(np.float32) + np.float32(1)
        assert len(np.unique(s32)) < G  # fp32 cannot tell them apart
    x = x.reshape(T, G * S)
    for by in ("max", "top2"):
        check(x, b, k, score, G, 3, by, "fp32")
        check(x, None, k, score, G, 3, by, "fp32")


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
def test_masks_and_non_finite(score, bias, by):
    E, G, k, inf = 40, 5, 4, np.inf
    rng = np.random.default_rng(1)
    x = rng.standard_normal((10, E)).astype(np.float32)
    low = np.finfo(np.float32).min
    x[0] = -inf                 # nothing selectable: the lowest groups and experts
    x[1, :] = -inf
    x[1, 17] = 0.5              # one expert left
    x[2, 5:] = low
    x[3] = low
    x[4, 7] = np.nan
    x[5, 8:16] = np.nan         # a whole group
    x[6] = np.nan
    x[7, 9] = inf
    x[8, [3, 30]] = inf
    x[9, ::2] = -inf
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    for top in (1, 2, 5):
        idx, w, x64 = run(x, b, k, score, 1, 1.0, G, top, by, "fp32")
        ridx, _ = B.grouped(x64, b, k, score, 1, 1.0, G, top, by)
        assert np.array_equal(idx, ridx), (top, idx, ridx)
        for row in idx:
            assert len(set(row)) == k and len(set(row // (E // G))) <= top
        # no number where NaN or, under softmax, +inf was selected
        taken = np.take_along_axis(x64, idx.astype(np.int64), axis=1)
        spoilt = np.isnan(taken).any(axis=1)
        if score == "softmax":
            spoilt |= np.isposinf(taken).any(axis=1)
        assert np.isnan(w[spoilt]).any(axis=1).all() and np.isfinite(w[~spoilt]).all()


@pytest.mark.parametrize("by", ["max", "top2"])
def test_biases_that_keep_out_or_put_first(by):
    T, E, G, k, inf = 50, 64, 8, 6, np.inf
    rng = np.random.default_rng(4)
    x = rng.standard_normal((T, E)).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    b[:16] = -inf                                # two groups kept out
    b[16] = np.finfo(np.float32).min
    b[33], b[60] = inf, 1e6
    b[40:44] = [3e38, 3e38, -3e38, np.nan]       # a sum past fp32, not past 64 bits
    for top in (1, 3, 7):
        check(x, b, k, "sigmoid", G, top, by, "bf16", weights=False)


def test_batches():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((16411, 64)).astype(np.float32)
    b = (rng.standard_normal(64) * 0.1).astype(np.float32)
    check(x, b, 6, "sigmoid", 8, 3, "top2", "bf16")
    cfg = M.MepGateConfig(64, 6, M.MEP_SCORE_SIGMOID, M.MEP_BF16, 1, 1.0, 0.0)
    M.mep_gate_grouped(cfg, 8, 3, M.MEP_GROUP_TOP2, None, None, 0, None, None)  # no tokens


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("E,G", [(24, 4), (256, 8), (1024, 16), (126, 42)])
def test_infinite_logits_beside_ones_past_exp(E, G, dtype, by):
    # a logit of +inf puts its group first, also among finite ones whose exponentials 64
    # bits do not hold; the groups behind it go by those
    S, k = E // G, 3
    rng = np.random.default_rng(E)
    x = rng.standard_normal((40, G, S)).astype(np.float32)
    for t in range(40):
        at = rng.permutation(G)
        x[t, at[0], rng.integers(S)] = np.inf
        x[t, at[1], :2] = (760.0, 750.0) if t % 4 else (3e38, 2e38)
        x[t, at[2], :2] = (768.0, 90.0) if t % 4 else (2.5e38, 2.25e38)
        if t % 5 == 1:
            x[t, at[1], 1] = np.inf
        if t % 5 == 2:
            x[t, at[1], 0] = np.nan
        if t % 5 == 3:
            x[t, at[0]][x[t, at[0]] < np.inf] = -np.inf
        if t == 39:
            x[t][x[t] < np.inf] = -np.inf    # nothing finite is left
    x = x.reshape(40, E)
    for top in (1, 2, 3):
        if top * S < k:
            continue
        idx, _, x64 = run(x, None, k, "softmax", 1, 1.0, G, top, by, dtype)
        of = np.where(np.isnan(x64), -np.inf, x64)
        if by == "top2":  # a softmax is the same of logits that are all less by one number
            largest = np.where(np.isfinite(x64), x64, -np.inf).max(axis=1, keepdims=True)
            of = np.exp(of - np.where(np.isfinite(largest), largest, 0.0))
        inside = -np.sort(-of.reshape(40, G, S), axis=2)
        best = inside[:, :, 0]
        if by == "top2":
            best = np.where(best == np.inf, best, best + inside[:, :, 1])
        chosen = R.top(best, top)
        for t in range(40):
            at = np.concatenate([np.arange(g * S, g * S + S) for g in sorted(chosen[t])])
            assert np.array_equal(idx[t], at[R.top(x64[t, at][None], k)[0]]), (top, t, idx[t])
            assert x64[t, idx[t, 0]] == np.inf
