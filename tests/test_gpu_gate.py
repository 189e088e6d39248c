"""Router, balance loss and their gradient against 64-bit references.

Tolerances count roundings (``_experts_ref.prob_steps``): every fp32 result is
a probability or a sum of products of probabilities, so it is held to that many
half-steps of fp32 relative to the magnitudes the formula adds up, and a bf16
result to half a step of bf16 more."""

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _experts_ref as R

pytestmark = pytest.mark.gpu

SCORE = {"softmax": M.MEP_SCORE_SOFTMAX, "sigmoid": M.MEP_SCORE_SIGMOID}
DTYPE = {"fp32": (M.MEP_FP32, torch.float32), "bf16": (M.MEP_BF16, torch.bfloat16)}


def cfg(E, k, score, dtype, normalize=1, scale=1.0, coef=0.02):
    return M.MepGateConfig(E, k, SCORE[score], DTYPE[dtype][0], normalize, scale, coef)


def make_logits(T, E, dtype, seed, spread=2.0):
    """Normal logits within +-12 (device tensor in the type, host fp64)."""
    rng = np.random.default_rng(seed)
    x = np.clip(rng.standard_normal((T, E)) * spread, -12, 12).astype(np.float32)
    t = torch.from_numpy(x).to(DTYPE[dtype][1])
    return t.cuda(), t.double().numpy()


def run_gate(c, logits, bias, T, stream=None):
    idx = torch.full((T + 1, c.top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, c.top_k), -7.0, device="cuda")
    M.mep_gate(c, logits, bias, T, idx, w, stream)
    torch.cuda.synchronize()
    assert bool((idx[T:] == -7).all()) and bool((w[T:] == -7).all())  # nothing behind the last row
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


def close(got, ref, mag, steps, dtype="fp32"):
    got = np.asarray(got, dtype=np.float64)
    tol = steps * R.U32 * mag + (R.UBF16 * np.abs(ref) if dtype == "bf16" else 0.0) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


SIZES = [(1, 1, 1), (1, 256, 8), (3, 8, 8), (5, 33, 32), (2, 64, 6), (257, 60, 4), (130, 65, 7),
         (77, 128, 3), (65, 129, 9), (1000, 256, 8), (33, 300, 17), (40, 512, 10), (19, 513, 8),
         (9, 1000, 32), (6, 1024, 5), (7, 1601, 12), (5, 4096, 32)]


@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gate(T, E, k, dtype, score, bias):
    logits, x = make_logits(T, E, dtype, T * 1000 + E)
    b = np.random.default_rng(5).standard_normal(E).astype(np.float32) * 0.2 if bias else None
    bt = torch.from_numpy(b).cuda() if bias else None
    for normalize, scale in ((1, 1.0), (0, 2.5)):
        idx, w = run_gate(cfg(E, k, score, dtype, normalize, scale), logits, bt, T)
        ridx, rw = R.gate(x, b, k, score, normalize, scale)
        assert np.array_equal(idx, ridx)
        close(w, rw, np.abs(rw), R.prob_steps())


@pytest.mark.parametrize("bias", ["none", "zero", "two values"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_ties_go_to_the_lowest_expert(score, bias):
    # logits from four values only: every selection is among equals
    T, E, k = 200, 100, 8
    if score == "softmax" and bias != "none":
        pytest.skip("a bias needs sigmoid scores")
    rng = np.random.default_rng(3)
    x = rng.choice([-1.5, 0.0, -0.0, 2.0], size=(T, E)).astype(np.float32)
    b = None if bias == "none" else np.zeros(E, np.float32)
    if bias == "two values":
        b[::3] = 0.125
    idx, _ = run_gate(cfg(E, k, score, "bf16"), torch.from_numpy(x).bfloat16().cuda(),
                      None if b is None else torch.from_numpy(b).cuda(), T)
    ridx, _ = R.gate(x, b, k, score, 1, 1.0)
    assert np.array_equal(idx, ridx)


def test_gate_orders_sigmoid_scores_closer_than_fp32_tells():
    # neighbouring logits one fp32 step apart around 3 and a bias of 1: the fp32
    # scores are equal in groups, their 64-bit values are not
    T, E, k = 64, 256, 8
    rng = np.random.default_rng(11)
    steps = np.stack([rng.permutation(E) for _ in range(T)])
    x = (np.float32(3.0) + steps.astype(np.float32) * np.float32(2 ** -22)).astype(np.float32)
    b = np.ones(E, np.float32)
    s32 = (1 / (1 + np.exp(-x))).astype(np.float32) + b
    assert len(np.unique(s32[0])) < E // 4  # fp32 cannot tell most of them apart
    idx, _ = run_gate(cfg(E, k, "sigmoid", "fp32"), torch.from_numpy(x).cuda(),
                      torch.from_numpy(b).cuda(), T)
    assert np.array_equal(idx, R.gate(x, b, k, "sigmoid", 1, 1.0)[0])
    # the border alone undecided, among equals and near equals
    x2 = np.full((4, 16), -5.0, np.float32)
    x2[:, 3], x2[:, 9], x2[:, 12] = 3.0, 3.0, np.float32(3.0) + np.float32(2 ** -22)
    idx, _ = run_gate(cfg(16, 1, "sigmoid", "fp32"), torch.from_numpy(x2).cuda(),
                      torch.ones(16, device="cuda"), 4)
    assert np.array_equal(idx, np.full((4, 1), 12))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
def test_gate_masked_and_non_finite_logits(score, normalize):
    E, k = 40, 4
    inf = np.inf
    x = np.random.default_rng(1).standard_normal((8, E)).astype(np.float32)
    x[0] = -inf                        # nothing selectable
    x[1, :] = -inf
    x[1, 17] = 0.5                     # one expert left
    x[2, 5:] = np.finfo(np.float32).min  # the type's lowest value
    x[3] = np.finfo(np.float32).min
    x[4, 7] = np.nan
    x[5, 9] = inf
    x[6] = np.nan
    idx, w = run_gate(cfg(E, k, score, "fp32", normalize), torch.from_numpy(x).cuda(), None, 8)
    assert ((idx >= 0) & (idx < E)).all()
    assert all(len(set(r)) == k for r in idx)
    good = [0, 1, 2, 3, 7]
    ridx, rw = R.gate(x[good], None, k, score, normalize, 1.0)
    assert np.array_equal(idx[good], ridx)
    close(w[good], rw, np.abs(rw), R.prob_steps())
    assert (w[0] == 0).all()
    assert 7 not in idx[4]             # NaN ranks last
    assert idx[5][0] == 9
    if score == "softmax":
        assert np.isnan(w[5]).all()
        assert np.isnan(w[4]).all() == (not normalize)
    else:
        assert np.isfinite(w[4]).all() and np.isfinite(w[5]).all()
    assert np.array_equal(idx[6], np.arange(k)) and np.isnan(w[6]).all()


def test_gate_no_tokens_and_rows_behind_the_last():
    c = cfg(256, 8, "softmax", "fp32")
    idx, w = run_gate(c, torch.zeros((1, 256), device="cuda"), None, 0)
    assert idx.shape == (0, 8)


def test_gate_offsets_past_32_bits():
    # 530000 x 4096 logits: the last rows lie past 2^31 elements
    T, E, k = 530000, 4096, 8
    assert T * E > 2 ** 31
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    last, x = make_logits(3, E, "bf16", 4)
    logits[T - 3:] = last
    c = cfg(E, k, "softmax", "bf16", 1, 1.0)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    M.mep_gate(c, logits, None, T, idx, w)
    gw = torch.zeros((T, k), device="cuda")
    gw[T - 3:] = 1.0 + torch.arange(k, device="cuda")
    out = torch.full((T, E), 3.0, dtype=torch.bfloat16, device="cuda")
    M.mep_gate_backward(c, logits, idx, None, T, gw, None, None, out)
    torch.cuda.synchronize()
    ridx, rw = R.gate(x, None, k, "softmax", 1, 1.0)
    assert np.array_equal(idx[T - 3:].cpu().numpy(), ridx)
    assert bool((idx[: T - 3] == torch.arange(k, device="cuda")).all())
    g, mag = R.gate_grad(x, ridx, None, "softmax", 1, 1.0, 0.02, gw[T - 3:].cpu().numpy(), None,
                         0.0)
    close(out[T - 3:].float().cpu().numpy(), g, mag, 2 * R.prob_steps(), "bf16")
    assert not bool(out[: T - 3].any())


BAL = [(1, 1, 1), (1, 256, 8), (37, 8, 2), (1021, 60, 4), (300, 65, 7), (4096, 256, 8),
       (70, 512, 10), (21, 1601, 12), (9, 4096, 32)]


def run_balance(c, logits, idx, mask, T, ws=None):
    E = c.num_experts
    counts = torch.full((E + 2,), -7, dtype=torch.int32, device="cuda")
    mean = torch.full((E + 1,), -7.0, device="cuda")
    loss = torch.full((1,), -7.0, device="cuda")
    if ws is None:
        ws = torch.zeros(M.mep_balance_workspace_bytes(c, T), dtype=torch.uint8, device="cuda")
    M.mep_balance_loss(c, logits, idx, mask, T, counts, mean, loss, ws)
    torch.cuda.synchronize()
    assert int(counts[E + 1]) == -7 and float(mean[E]) == -7.0
    return counts[: E + 1].cpu().numpy(), mean[:E].cpu().numpy(), float(loss[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", BAL)
def test_balance(T, E, k, masked, dtype, score):
    logits, x = make_logits(T, E, dtype, T + E)
    idx = R.top(x, k)
    rng = np.random.default_rng(T)
    if T > 2:
        idx[1, 0] = -1        # a dropped position
        idx[2, k - 1] = E     # an id out of range
        idx[0, :] = idx[0, 0]  # one expert named k times
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    if masked and T > 1:      # padding may hold anything
        mask[T // 2] = 0
        logits[T // 2] = float("nan")
    c = cfg(E, k, score, dtype)
    got = run_balance(c, logits, torch.from_numpy(idx).cuda(),
                      None if mask is None else torch.from_numpy(mask).cuda(), T)
    ref = R.balance(x, idx, mask, score, 0.02)
    assert np.array_equal(got[0], ref[0])
    # a group of lanes adds up its tokens one by one, 8 to 32 groups join
    # in order, and blocks in 64 bits
    steps = R.prob_steps() + T / 4 + 34
    close(got[1], ref[1], ref[1], steps)
    close(np.float64(got[2]), np.float64(ref[2]), np.float64(ref[2]), steps + 2)


def test_balance_nothing_counts():
    c = cfg(60, 4, "softmax", "fp32")
    nan = torch.full((5, 60), float("nan"), device="cuda")
    idx = torch.zeros((5, 4), dtype=torch.int32, device="cuda")
    mask = torch.zeros(5, dtype=torch.uint8, device="cuda")
    for T, m in ((0, None), (5, mask)):
        counts, mean, loss = run_balance(c, nan, idx, m, T)
        assert not counts.any() and not mean.any() and loss == 0.0
    # and its gradient is zero, without a division by the count
    out = torch.full((5, 60), 7.0, device="cuda")
    M.mep_gate_backward(c, torch.zeros((5, 60), device="cuda"), idx, None, 5, None,
                        torch.zeros(61, dtype=torch.int32, device="cuda"),
                        torch.ones(1, device="cuda"), out)
    assert not bool(out.any())


def test_balance_all_minus_infinity_row_adds_nothing():
    c = cfg(16, 2, "softmax", "fp32")
    x = torch.full((2, 16), float("-inf"), device="cuda")
    x[1] = 0.0
    idx = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    counts, mean, _ = run_balance(c, x, idx, None, 2)
    assert counts[0] == 4 and np.array_equal(mean, np.full(16, 1 / 32, np.float32))


def test_balance_workspace_serves_calls_in_turn_and_results_repeat():
    c = cfg(256, 8, "softmax", "fp32")
    ws = torch.zeros(M.mep_balance_workspace_bytes(c, 4096), dtype=torch.uint8, device="cuda")
    seen = {}
    for turn in range(3):
        for T in (4096, 100, 1):
            logits, x = make_logits(T, 256, "fp32", T)
            idx = torch.from_numpy(R.top(x, 8)).cuda()
            got = run_balance(c, logits, idx, None, T, ws)
            if turn == 0:
                seen[T] = got
            assert np.array_equal(got[0], seen[T][0]) and np.array_equal(got[1], seen[T][1])
            assert got[2] == seen[T][2]  # bit for bit: no order of its own


GRAD = [(1, 1, 1), (1, 256, 8), (5, 33, 32), (257, 60, 4), (130, 65, 7), (500, 256, 8),
        (40, 512, 10), (19, 513, 8), (7, 1601, 12), (5, 4096, 32)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,k", GRAD)
def test_gate_backward(T, E, k, dtype, normalize, score):
    logits, x = make_logits(T, E, dtype, 3 * T + E)
    idx = R.top(x, k)
    rng = np.random.default_rng(T)
    if T > 3:
        idx[1, 0] = -1
        idx[2, k - 1] = E + 5
        idx[3, :] = idx[3, 0]          # one expert k times
    gw = rng.standard_normal((T, k)).astype(np.float32)
    mask = np.ones(T, np.uint8)
    if T > 4:
        mask[4] = 0
        logits[4] = float("nan")
    counts = R.balance(x, idx, mask, score, 0.02)[0].astype(np.int32)
    c = cfg(E, k, score, dtype, normalize, 1.5)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        out = torch.full((T + 1, E), 7.0, dtype=DTYPE[dtype][1], device="cuda")
        M.mep_gate_backward(c, logits, dev(idx), dev(mask), T, dev(gw) if use_w else None,
                            dev(counts) if use_l else None,
                            torch.full((1,), 30.0, device="cuda") if use_l else None, out)
        torch.cuda.synchronize()
        assert bool((out[T:] == 7.0).all())
        ref, mag = R.gate_grad(x, idx, mask, score, normalize, 1.5, 0.02, gw if use_w else None,
                               counts if use_l else None, 30.0)
        # a product of two probabilities, and the sums over a token's experts
        close(out[:T].float().cpu().numpy(), ref, mag, 3 * R.prob_steps(), dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
def test_gate_backward_against_differences(score, normalize):
    # central differences of the 64-bit weights and loss: step 1e-5, so the
    # truncation (h^2/6 times a third derivative of order one) is below 1e-9 and
    # the cancellation about 1e-16 / 1e-5
    T, E, k = 4, 20, 3
    logits, x = make_logits(T, E, "fp32", 9, 1.0)
    idx = R.top(x, k)
    rng = np.random.default_rng(2)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    counts, _, _ = R.balance(x, idx, None, score, 0.02)
    gl = 25.0

    def value(q):
        return (R.gate_weights(q, idx, score, normalize, 1.5) * gw).sum() + \
            gl * R.balance(q, idx, None, score, 0.02)[2]

    num, h = np.zeros((T, E)), 1e-5
    for t in range(T):
        for e in range(E):
            a, b = x.copy(), x.copy()
            a[t, e] += h
            b[t, e] -= h
            num[t, e] = (value(a) - value(b)) / (2 * h)
    out = torch.empty((T, E), device="cuda")
    M.mep_gate_backward(cfg(E, k, score, "fp32", normalize, 1.5), logits,
                        torch.from_numpy(idx).cuda(), None, T, torch.from_numpy(gw).cuda(),
                        torch.from_numpy(counts.astype(np.int32)).cuda(),
                        torch.full((1,), gl, device="cuda"), out)
    _, mag = R.gate_grad(x, idx, None, score, normalize, 1.5, 0.02, gw, counts, gl)
    assert np.all(np.abs(out.cpu().numpy() - num) <= 3 * R.prob_steps() * R.U32 * mag + 1e-8)
