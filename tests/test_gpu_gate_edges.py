"""The router where its number formats end: ties that outnumber a lane's
registers, logits far below zero, the largest batch.

Half-steps of fp32 (2^-24, relative) of a result below: an exponential 4 (the
hardware's within one unit of the last place, two products and a sum), of a
difference to the largest logit one for each unit of that difference; 1 + e, its
reciprocal (2) and a product 4, so a score is within 8 + spread of its value; a
sum of n of them n more; a quotient 2."""

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _experts_ref as R
from test_gpu_gate import cfg, close, run_balance, run_gate

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# (experts, k): k below, at and above the number of values that a lane holds
TIES = [(64, 9), (64, 10), (64, 32), (60, 12), (8, 8), (33, 32), (128, 8), (128, 10), (128, 32),
        (100, 11), (256, 17), (256, 32), (130, 20), (300, 32), (1024, 17), (1024, 32), (513, 25),
        (4096, 32)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("E,k", TIES)
def test_biased_ties(E, k, dtype):
    rng = np.random.default_rng(E + k)
    x = np.zeros((40, E), np.float32)
    x[1, 5] = 1.0                                    # one above an equal row
    x[2, [0, E // 2, E - 1]] = 1.0, 2.0, 0.5         # a few, all different
    x[3, : E // 2] = 1.0                             # two values
    x[4] = -np.inf
    x[5, 1:] = -np.inf
    x[6, ::3] = -np.inf
    x[7, 2] = -1.0                                   # one below
    for t in range(8, 24):                           # few values, many equals
        x[t] = rng.choice(np.float32([0.0, 0.5, -2.0]), size=E, p=[0.9, 0.05, 0.05])
    for t in range(24, 40):                          # a handful above, the rest equal
        at = rng.choice(E, size=min(E, 1 + t % 7), replace=False)
        x[t, at] = 1.0 + np.arange(len(at), dtype=np.float32)
    bias = np.zeros(E, np.float32)
    for name in ("zero", "two values", "one"):
        b = bias.copy()
        if name == "two values":
            b[::4] = 0.25
        elif name == "one":
            b[E // 3] = 0.125
        idx, w = run_gate(cfg(E, k, "sigmoid", dtype), torch.from_numpy(x).to(DTYPES[dtype]).cuda(),
                          torch.from_numpy(b).cuda(), len(x))
        assert all(len(set(r)) == k for r in idx.tolist()), (name, "an expert twice")
        ridx, rw = R.gate(x, b, k, "sigmoid", 1, 1.0)
        assert np.array_equal(idx, ridx), (name, np.argwhere((idx != ridx).any(1))[:4])
        close(w, rw, np.abs(rw), R.prob_steps())


def scores_far_from_zero(T, E, seed, lo=20.0, hi=80.0):
    """Logits of both signs with magnitudes in [lo, hi], eighths (so exact in
    bf16's and fp32's products with small numbers of them)."""
    rng = np.random.default_rng(seed)
    x = rng.integers(int(8 * lo), int(8 * hi), size=(T, E)) / 8.0
    return (x * rng.choice([-1.0, 1.0], size=(T, E))).astype(np.float32)


@pytest.mark.parametrize("E,k", [(16, 16), (100, 32), (256, 32), (1030, 32)])
def test_sigmoid_weights_far_below_zero(E, k):
    # every selected logit is far below zero: the error of its exponential must
    # not grow with its size
    x = -np.abs(scores_far_from_zero(50, E, E))
    idx, w = run_gate(cfg(E, k, "sigmoid", "fp32", 0, 2.5), torch.from_numpy(x).cuda(), None, 50)
    ridx, rw = R.gate(x, None, k, "sigmoid", 0, 2.5)
    assert np.array_equal(idx, ridx)
    close(w, rw, rw, 8 + 2)          # the score, times the scale (itself exact)
    g = np.random.default_rng(1).standard_normal((50, k)).astype(np.float32)
    out = torch.empty((50, E), device="cuda")
    M.mep_gate_backward(cfg(E, k, "sigmoid", "fp32", 0, 2.5), torch.from_numpy(x).cuda(),
                        torch.from_numpy(ridx).cuda(), None, 50, torch.from_numpy(g).cuda(), None,
                        None, out)
    ref, mag = R.gate_grad(x, ridx, None, "sigmoid", 0, 2.5, 0.0, g, None, 0.0)
    close(out.cpu().numpy(), ref, mag, 4 + 2 * 4 + 4)  # e / (1 + e)^2 times grad times scale


def test_softmax_weights_far_below_the_largest():
    # eighths: the difference to the largest logit is exact
    x = scores_far_from_zero(50, 8, 3, 0.0, 40.0)
    idx, w = run_gate(cfg(8, 8, "softmax", "fp32", 0, 2.5), torch.from_numpy(x).cuda(), None, 50)
    ridx, rw = R.gate(x, None, 8, "softmax", 0, 2.5)
    assert np.array_equal(idx, ridx)
    # numerator 4, 8 exponentials of 4 and their sum 8, quotient and scale 2
    close(w, rw, rw, 4 + 4 + 8 + 2)


# Where all that count are so far below zero that fp32 has no sigmoid for them
# (under -87.3), what is normalized is still well defined.
LOW = [(-100.0, -90.0), (-700.0, -690.0), (-110.0, -60.0), (-30.0, -12.0),
       (-3000.0, -2990.0)]  # the last vanish in 64 bits too: all weights are 0


@pytest.mark.parametrize("lo,hi", LOW)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,k", [(16, 4), (256, 8), (1030, 32)])
def test_normalized_sigmoid_weights_of_very_low_logits(E, k, bias, lo, hi):
    T, rng = 30, np.random.default_rng(E)
    x = rng.uniform(lo, hi, size=(T, E)).astype(np.float32)
    x[3, 1:] = -np.inf
    x[4] = -np.inf
    # experts that a bias selects, wherever their logits lie
    b = None if not bias else (rng.permutation(E) / 64.0).astype(np.float32)
    c = cfg(E, k, "sigmoid", "fp32", 1, 1.5)
    idx, w = run_gate(c, torch.from_numpy(x).cuda(), None if b is None else torch.from_numpy(b).cuda(), T)
    ridx, rw = R.gate(x, b, k, "sigmoid", 1, 1.5)
    assert np.array_equal(idx, ridx)
    # twice a score (8, and a step for each unit of difference), the sum, two more
    close(w, rw, rw, 2 * (8 + hi - lo) + k + 2)
    assert np.allclose(w[:3].sum(1), 1.5 if lo > -708 else 0.0) and (w[4] == 0).all()


@pytest.mark.parametrize("lo,hi", LOW)
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("E,k", [(16, 4), (256, 8), (1030, 32)])
def test_loss_and_gradients_of_very_low_sigmoid_logits(E, k, normalize, lo, hi):
    T, rng = 30, np.random.default_rng(E)
    x = rng.uniform(lo, hi, size=(T, E)).astype(np.float32)
    x[3, 1:] = -np.inf
    x[4] = -np.inf
    x[5, 1:] = 2.0                   # one row as usual
    idx = R.top(x, k)
    c = cfg(E, k, "sigmoid", "fp32", normalize, 1.5)
    xt, it = torch.from_numpy(x).cuda(), torch.from_numpy(idx).cuda()
    counts, mean, loss = run_balance(c, xt, it, None, T)
    ref = R.balance(x, idx, None, "sigmoid", 0.02)
    assert np.array_equal(counts, ref[0])
    # scores 8, a step for each unit of difference, a lane's sum and the lanes', the tokens'
    steps = 2 * (8 + hi - lo) + 70 + T + 4
    close(mean, ref[1], ref[1], steps)
    close(np.float64(loss), np.float64(ref[2]), np.float64(ref[2]), steps + 2)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.empty((T, E), device="cuda")
    M.mep_gate_backward(c, xt, it, None, T, torch.from_numpy(gw).cuda(),
                        torch.from_numpy(counts).cuda(), torch.full((1,), 30.0, device="cuda"), out)
    g, mag = R.gate_grad(x, idx, None, "sigmoid", normalize, 1.5, 0.02, gw, counts, 30.0)
    close(out.cpu().numpy(), g, mag, 3 * steps)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [40.0, 95.0, 150.0])
@pytest.mark.parametrize("E,k", [(16, 4), (256, 8), (1030, 32)])
def test_gradient_of_normalized_weights_for_experts_far_from_the_largest(E, k, far, score):
    # indices of an earlier routing, replayed on logits whose largest lies elsewhere
    T, rng = 20, np.random.default_rng(E)
    x = rng.uniform(-5, 0, size=(T, E)).astype(np.float32)
    idx = np.stack([rng.choice(np.arange(1, E), size=k, replace=False) for _ in range(T)])
    idx = idx.astype(np.int32)
    np.put_along_axis(x, idx.astype(np.int64), rng.uniform(-far - 4, -far, size=(T, k)).astype(np.float32), 1)
    x[:, 0] = 3.0
    idx[1, 0] = -1                   # a dropped position
    idx[2, 0] = idx[2, 1]            # an expert twice
    idx[3] = -1                      # no position left
    gw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.empty((T, E), device="cuda")
    M.mep_gate_backward(cfg(E, k, score, "fp32", 1, 1.5), torch.from_numpy(x).cuda(),
                        torch.from_numpy(idx).cuda(), None, T, torch.from_numpy(gw).cuda(), None,
                        None, out)
    ref, mag = R.gate_grad(x, idx, None, score, 1, 1.5, 0.0, gw, None, 0.0)
    assert np.abs(ref[4:]).max() > 0.01
    # three quotients of scores (8, and a step for each unit of their difference) and
    # sums of k, and the differences that the magnitudes cover
    close(out.cpu().numpy(), ref, mag, 3 * (8 + 5 + k + 4))


def test_largest_batch():
    # 2^26 tokens with 64 lanes each are 2^32 threads, one more than a launch takes
    T, E, k = 1 << 26, 513, 2
    torch.cuda.empty_cache()
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, T - 2, T - 1])
    x = np.random.default_rng(0).standard_normal((len(at), E)).astype(np.float32)
    x = torch.from_numpy(x).bfloat16()
    logits[at.cuda()] = x.cuda()
    c = cfg(E, k, "softmax", "bf16", 1, 1.0)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    M.mep_gate(c, logits, None, T, idx, w)
    ridx, rw = R.gate(x.double().numpy(), None, k, "softmax", 1, 1.0)
    assert np.array_equal(idx[at.cuda()].cpu().numpy(), ridx)
    close(w[at.cuda()].cpu().numpy(), rw, rw, R.prob_steps())
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[at.cuda()] = False
    assert bool(((idx == torch.arange(k, device="cuda", dtype=torch.int32)).all(1) | ~others).all())
    assert bool(((w == 0.5).all(1) | ~others).all())
    gw = torch.zeros((T, k), device="cuda")
    gw[at.cuda()] = torch.tensor([1.0, -2.0], device="cuda")
    out = torch.full((T, E), 3.0, dtype=torch.bfloat16, device="cuda")
    M.mep_gate_backward(c, logits, idx, None, T, gw, None, None, out)
    g, mag = R.gate_grad(x.double().numpy(), ridx, None, "softmax", 1, 1.0, 0.0,
                         gw[at.cuda()].cpu().numpy(), None, 0.0)
    close(out[at.cuda()].float().cpu().numpy(), g, mag, 3 * R.prob_steps(), "bf16")
    step = 1 << 22
    for t in range(0, T, step):
        assert not bool((out[t:t + step].any(1) & others[t:t + step]).any())
    del logits, out
    torch.cuda.empty_cache()


def test_a_torch_without_the_bare_stream_query(monkeypatch):
    # the private handle that the binding prefers may go away
    if hasattr(torch._C, "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    x = np.random.default_rng(0).standard_normal((5, 64)).astype(np.float32)
    idx, _ = run_gate(cfg(64, 4, "softmax", "fp32"), torch.from_numpy(x).cuda(), None, 5)
    assert np.array_equal(idx, R.gate(x, None, 4, "softmax", 1, 1.0)[0])


@pytest.mark.parametrize("E,k", [(16, 6), (64, 12), (256, 8), (1030, 20)])
def test_experts_masked_by_their_bias(E, k):
    # -inf or the lowest value keeps an expert out while others are left, +inf
    # puts it first, NaN last; k of them all are named all the same
    T, rng = 20, np.random.default_rng(E)
    x = rng.standard_normal((T, E)).astype(np.float32)
    low = np.finfo(np.float32).min
    for value, left in ((-np.inf, E - 3), (-np.inf, k), (-np.inf, k - 2), (low, k - 2), (np.nan, k - 2),
                        (np.inf, 2), (np.inf, E - k - 1), (low, 1), (np.nan, 0), (-np.inf, 0)):
        b = rng.uniform(-0.5, 0.5, size=E).astype(np.float32)
        b[rng.choice(E, size=E - left, replace=False)] = value
        idx, w = run_gate(cfg(E, k, "sigmoid", "fp32", 0), torch.from_numpy(x).cuda(),
                          torch.from_numpy(b).cuda(), T)
        ridx, rw = R.gate(x, b, k, "sigmoid", 0, 1.0)
        assert all(len(set(r)) == k for r in idx.tolist()), (value, left)
        assert np.array_equal(idx, ridx), (value, left)
        close(w, rw, rw, 8 + 2)
