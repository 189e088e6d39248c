"""The experts' product and its gradients against 64-bit references.

Bound of a result: half a step of bf16 for its one rounding, plus the fp32
accumulation, at most one half-step of fp32 for each of the summed products
relative to the sum of their magnitudes, carried through the activation (slopes
below 1.13), plus the activation's own evaluation, 8 half-steps of fp32 of its
value."""

import math

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _experts_ref as R

pytestmark = pytest.mark.gpu

ACT = {"none": M.MEP_ACT_NONE, "gelu": M.MEP_ACT_GELU, "silu": M.MEP_ACT_SILU,
       "silu_glu": M.MEP_ACT_SILU_GLU}
SENT = 0x5A5A


def nz(N, act):
    return 2 * N if act == "silu_glu" else N


def layout(counts, extra=0):
    """Segment starts padded to 128 rows, and a capacity with `extra` rows behind."""
    counts = np.asarray(counts)
    off = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    return counts.astype(np.int32), off.astype(np.int32), int(off[-1]) + extra


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()


class Case:
    """Seeded inputs of one product; rows outside the counts are NaN, so a use
    of one shows."""

    def __init__(self, counts, K, N, act, bias=True, residual=True, fp8=False, seed=0, extra=0,
                 cap=None):
        rng = np.random.default_rng(seed)
        self.counts, self.off, self.cap = layout(counts, extra)
        if cap is not None:
            self.cap = cap
        E = self.E = len(counts)
        self.K, self.N, self.Nz, self.act, self.fp8 = K, N, nz(N, act), act, fp8
        self.used = np.zeros(self.cap, bool)
        for e in range(E):
            self.used[self.off[e]: min(self.off[e] + self.counts[e], self.cap)] = True
        x = rng.standard_normal((self.cap, K)).astype(np.float32)
        w = (rng.standard_normal((E, self.Nz, K)) / math.sqrt(K)).astype(np.float32)
        self.xs = self.ws = None
        if fp8:
            f8 = torch.float8_e4m3fn
            self.x = torch.from_numpy(x * 100).clamp(-448, 448).to(f8)
            self.w = torch.from_numpy(w * (100 * math.sqrt(K))).clamp(-448, 448).to(f8)
            xs = (rng.random((self.cap, K // 128)) + 0.5) / 100
            ws = (rng.random((E, self.Nz // 128, K // 128)) + 0.5) / (100 * math.sqrt(K))
            self.xs, self.ws = (torch.from_numpy(a.astype(np.float32)) for a in (xs, ws))
            self.x64 = self.x.double().numpy() * np.repeat(self.xs.double().numpy(), 128, axis=1)
            self.w64 = self.w.double().numpy() * np.repeat(np.repeat(
                self.ws.double().numpy(), 128, axis=1), 128, axis=2)
            self.x.view(torch.uint8)[~torch.from_numpy(self.used)] = 0x7F  # NaN
            self.xs[~torch.from_numpy(self.used)] = float("nan")
        else:
            self.x, self.w = bf16(x), bf16(w)
            self.x64, self.w64 = self.x.double().numpy(), self.w.double().numpy()
            self.x[~torch.from_numpy(self.used)] = float("nan")
        self.bias = rng.standard_normal((E, self.Nz)).astype(np.float32) if bias else None
        self.res = bf16(rng.standard_normal((self.cap, N))) if residual else None
        self.rng = rng
        self.cfg = M.MepLinearConfig(E, K, N, ACT[act], M.MEP_QUANT_FP8_E4M3_BLOCK128 if fp8
                                     else M.MEP_QUANT_NONE)

    def segments(self):
        for e in range(self.E):
            a, b = int(self.off[e]), int(min(self.off[e] + self.counts[e], self.cap))
            if b > a:
                yield e, a, b

    def dev(self, t):
        if t is None:
            return None
        return (t if torch.is_tensor(t) else torch.from_numpy(t)).cuda()

    def forward(self, num_rows=None, want_z=False):
        y = torch.full((self.cap, self.N), SENT, dtype=torch.int16, device="cuda")
        z = torch.full((self.cap, self.Nz), SENT, dtype=torch.int16, device="cuda") \
            if want_z else None
        n = int(self.counts.sum()) if num_rows is None else num_rows
        M.mep_expert_linear(self.cfg, self.dev(self.x), self.dev(self.xs), self.dev(self.counts),
                            self.dev(self.off), self.cap, n, self.dev(self.w), self.dev(self.ws),
                            self.dev(self.bias), self.dev(self.res), y, z)
        torch.cuda.synchronize()
        unused = torch.from_numpy(~self.used)
        for t in (y, z):
            if t is not None:
                assert bool((t.cpu()[unused] == SENT).all()), "a row outside the segments is written"
        got = y.view(torch.bfloat16).double().cpu().numpy()
        return got, None if z is None else z.view(torch.bfloat16).double().cpu().numpy()

    def lost_in_groups(self, e, a, b):
        """E4M3: the matrix instruction adds 8 neighbouring products on a grid of
        2^-13 of the largest one's power of two (of a product beside one of 2^16 in
        its group, nothing below 2^3 arrives; in another group, all down to fp32's
        2^-7).  The largest has 8 bits, so it lies on the grid; the 7 others lose
        less than a step each, 7 * 2^-13 of the largest, times the scales."""
        x, w = np.abs(self.x64[a:b]), np.abs(self.w64[e])
        lost = np.zeros((b - a, self.Nz))
        for k in range(0, self.K, 8):
            largest = np.zeros_like(lost)
            for q in range(k, k + 8):
                np.maximum(largest, np.outer(x[:, q], w[:, q]), out=largest)
            lost += 7 * 2.0 ** -13 * largest
        return lost

    def check_forward(self, **kw):
        got, z = self.forward(**kw)
        for e, a, b in self.segments():
            x, w = self.x64[a:b], self.w64[e]
            ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
            if self.bias is not None:
                ref, mag = ref + self.bias[e].astype(np.float64), mag + np.abs(self.bias[e])
            err = (self.K + 2) * R.U32 * mag
            if self.fp8:
                err = err + self.lost_in_groups(e, a, b)
            if z is not None:
                assert np.all(np.abs(z[a:b] - ref) <= err + R.UBF16 * (np.abs(ref) + err)), "z"
            y = R.act(ref, self.act, self.N)
            if self.act == "silu_glu":
                g, u = ref[:, : self.N], ref[:, self.N:]
                eg, eu = err[:, : self.N], err[:, self.N:]
                s = np.abs(R.act(g, "silu", self.N))
                err = 1.13 * eg * (np.abs(u) + eu) + (s + 1.13 * eg) * eu
            else:
                err = 1.13 * err
            err = err + 8 * R.U32 * np.abs(y)
            if self.res is not None:
                y = y + self.res[a:b].double().numpy()
                err = err + R.U32 * np.abs(y)
            bad = ~(np.abs(got[a:b] - y) <= err + R.UBF16 * (np.abs(y) + err))
            assert not bad.any(), (e, int(bad.sum()), np.argwhere(bad)[:4], got[a:b][bad][:4],
                                   y[bad][:4])

    def backward(self, wants=("x", "w", "b"), num_rows=None):
        gy = bf16(self.rng.standard_normal((self.cap, self.N)))
        z = bf16(self.rng.standard_normal((self.cap, self.Nz)) * 2) if self.act != "none" else None
        self.gy64 = gy.double().numpy()
        self.z64 = None if z is None else z.double().numpy()
        gy[~torch.from_numpy(self.used)] = float("nan")
        out = {"x": torch.full((self.cap, self.K), SENT, dtype=torch.int16, device="cuda"),
               "w": torch.full((self.E, self.Nz, self.K), SENT, dtype=torch.int16, device="cuda"),
               "b": torch.full((self.E, self.Nz), 7.0, device="cuda")}
        ws = torch.full((M.mep_linear_workspace_bytes(self.cfg, self.cap),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        n = int(self.counts.sum()) if num_rows is None else num_rows
        M.mep_expert_linear_backward(
            self.cfg, self.dev(gy), self.dev(z), self.dev(self.x), self.dev(self.w),
            self.dev(self.counts), self.dev(self.off), self.cap, n,
            *(out[q] if q in wants else None for q in "xwb"), ws)
        torch.cuda.synchronize()
        return out

    def check_backward(self, wants=("x", "w", "b"), **kw):
        out = self.backward(wants, **kw)
        unused = torch.from_numpy(~self.used)
        if "x" in wants:
            assert bool((out["x"].cpu()[unused] == SENT).all()), "a row outside is written"
        gx = out["x"].view(torch.bfloat16).double().cpu().numpy()
        gw = out["w"].view(torch.bfloat16).double().cpu().numpy()
        gb = out["b"].double().cpu().numpy()
        rounded = 0.0 if self.act == "none" else R.UBF16  # grad_z for the products
        have = {e: (a, b) for e, a, b in self.segments()}
        for e in range(self.E):
            if e not in have:
                assert "w" not in wants or not gw[e].any()
                assert "b" not in wants or not gb[e].any()
                continue
            a, b = have[e]
            z = None if self.z64 is None else self.z64[a:b]
            gz = R.act_grad(self.gy64[a:b], z, self.act, self.N)
            x, w = self.x64[a:b], self.w64[e]
            # grad_z: its evaluation is within 16 half-steps of fp32 of
            # |grad_y| (1 + |z|) (both halves), which covers cancelling slopes
            own = np.zeros_like(gz)
            if self.act != "none":
                m = np.abs(self.gy64[a:b])
                if self.act == "silu_glu":
                    g, u = z[:, : self.N], z[:, self.N:]
                    own = np.concatenate([m * np.abs(u) * (1 + np.abs(g)), m * np.abs(g)], axis=1)
                else:
                    own = m * (1 + np.abs(z))
            dz = 16 * R.U32 * own
            for name, got, ref, mag, more, steps in (
                    ("x", gx[a:b], gz @ w, np.abs(gz) @ np.abs(w), dz @ np.abs(w), self.Nz),
                    ("w", gw[e], gz.T @ x, np.abs(gz).T @ np.abs(x), dz.T @ np.abs(x), b - a)):
                if name not in wants:
                    continue
                err = (rounded + (steps + 2) * R.U32) * mag + (1 + rounded) * more
                bad = ~(np.abs(got - ref) <= err + R.UBF16 * (np.abs(ref) + err))
                assert not bad.any(), (name, e, int(bad.sum()), np.argwhere(bad)[:4],
                                       got[bad][:4], ref[bad][:4])
            if "b" in wants:
                # a wave adds 16 rows one by one, eight waves join; blocks in 64 bits
                err = 36 * R.U32 * np.abs(gz).sum(0) + dz.sum(0)
                assert np.all(np.abs(gb[e] - gz.sum(0)) <= err + R.U32 * np.abs(gb[e])), "bias"


COUNTS = {"one row": [1], "one segment": [200], "gaps": [0, 3, 0, 0, 130, 1, 0],
          "full": [128, 256], "skewed": [2, 700, 0, 17], "many": [1, 2, 0, 5] * 20,
          "nothing": [0, 0, 0]}


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("name", list(COUNTS))
def test_forward(name, act):
    Case(COUNTS[name], 136, 72, act, extra=5).check_forward(want_z=True)


@pytest.mark.parametrize("K,N", [(8, 8), (64, 16), (72, 200), (512, 128), (1048, 264), (2048, 64)])
@pytest.mark.parametrize("act", ["none", "silu_glu"])
def test_forward_sizes(K, N, act):
    Case([3, 150, 0, 40], K, N, act, bias=False, residual=False).check_forward()


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("name", list(COUNTS))
def test_forward_fp8(name, act):
    Case(COUNTS[name], 256, 128, act, fp8=True, extra=3).check_forward(want_z=True)


@pytest.mark.parametrize("K,N", [(128, 128), (384, 256), (1024, 384)])
def test_forward_fp8_sizes(K, N):
    Case([3, 150, 0, 40], K, N, "silu_glu", bias=False, residual=False, fp8=True).check_forward()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_rows", [0, 1, 20, 5000, 10 ** 9])
def test_num_rows_changes_no_result(num_rows, fp8):
    # whatever the caller expects, every row of every segment is computed
    Case([300, 0, 5, 64, 129], 256, 128, "gelu", fp8=fp8, extra=700).check_forward(
        num_rows=num_rows, want_z=True)


@pytest.mark.parametrize("num_rows", [0, 10 ** 9])
@pytest.mark.parametrize("K", [64, 128, 192, 200, 256, 320, 456])
def test_forward_depths(K, num_rows):
    # odd and even numbers of steps, with and without a rest, in both tile sizes
    Case([300, 0, 5], K, 136, "silu_glu", extra=1).check_forward(num_rows=num_rows, want_z=True)


@pytest.mark.parametrize("num_rows", [0, 10 ** 9])
@pytest.mark.parametrize("K", [128, 256, 384, 640])
def test_forward_depths_fp8(K, num_rows):
    Case([300, 0, 5], K, 128, "silu_glu", fp8=True, extra=1).check_forward(num_rows=num_rows)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K,N", [(128, 128), (384, 128), (1024, 256)])
def test_single_rows(K, N, fp8):
    # few rows: the summed index split over waves, some without a part of it
    for act in ("none", "silu_glu"):
        Case([1, 0, 2, 17, 1], K, N, act, fp8=fp8).check_forward(num_rows=21, want_z=True)


@pytest.mark.parametrize("num_rows", [0, 10 ** 9])
def test_most_experts(num_rows):
    counts = [0] * 4096
    for e, n in ((0, 3), (63, 1), (64, 129), (2000, 2), (4095, 260)):
        counts[e] = n
    Case(counts, 24, 16, "silu_glu").check_forward(num_rows=num_rows, want_z=True)
    Case(counts, 24, 16, "silu_glu").check_backward(num_rows=num_rows)


def test_many_experts_fp8():
    counts = [0] * 600
    for e, n in ((1, 3), (300, 300), (599, 1)):
        counts[e] = n
    Case(counts, 128, 128, "none", fp8=True).check_forward(num_rows=10 ** 9)


def test_rows_past_the_capacity_are_left_out():
    Case([100, 200, 50], 64, 32, "silu", cap=128 + 130).check_forward()
    Case([100, 200, 50], 64, 32, "silu", cap=128 + 130).check_backward()
    Case([100, 200, 50], 64, 32, "none", cap=128).check_backward()


def test_residual_in_place():
    c = Case([40, 0, 150], 64, 48, "silu")
    ref, _ = c.forward()
    y = c.res.cuda()
    M.mep_expert_linear(c.cfg, c.dev(c.x), None, c.dev(c.counts), c.dev(c.off), c.cap, 190,
                        c.dev(c.w), None, c.dev(c.bias), y, y, None)
    assert np.array_equal(y.double().cpu().numpy()[c.used], ref[c.used])


@pytest.mark.parametrize("counts,num_rows", [([1, 0, 2], 3), ([300, 0, 5], 10 ** 9)])
@pytest.mark.parametrize("act", ["none", "silu_glu"])
def test_residual_in_place_few_rows_and_large_tiles(counts, num_rows, act):
    c = Case(counts, 192, 136, act)
    ref, _ = c.forward(num_rows=num_rows)
    y = c.res.cuda()
    M.mep_expert_linear(c.cfg, c.dev(c.x), None, c.dev(c.counts), c.dev(c.off), c.cap, num_rows,
                        c.dev(c.w), None, c.dev(c.bias), y, y, None)
    assert np.array_equal(y.double().cpu().numpy()[c.used], ref[c.used])


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("name", list(COUNTS))
def test_backward(name, act):
    Case(COUNTS[name], 136, 72, act, extra=5).check_backward()


@pytest.mark.parametrize("K,N", [(8, 8), (64, 16), (72, 200), (512, 128), (1048, 264)])
@pytest.mark.parametrize("act", ["none", "silu_glu"])
def test_backward_sizes(K, N, act):
    Case([3, 150, 0, 40], K, N, act).check_backward()


@pytest.mark.parametrize("N", [64, 128, 192, 200, 320, 456])
def test_backward_depths(N):
    # grad_x sums over N: odd and even numbers of steps, large tiles
    Case([300, 0, 5], 264, N, "none", extra=1).check_backward(num_rows=10 ** 9)


def test_backward_large_tiles():
    # enough 256 x 256 tiles of grad_w that it takes them: 40 x 3 x 3; lengths of
    # no, one and several steps, with rests of every kind
    counts = [0, 1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 256, 300, 320, 8, 0] + [5, 70] * 12
    Case(counts, 520, 264, "silu_glu", extra=3).check_backward(num_rows=10 ** 9)


@pytest.mark.parametrize("wants", [("x",), ("w",), ("b",), ("x", "b"), ("w", "b")])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_parts(wants, act):
    c = Case([3, 150, 0, 40], 72, 40, act)
    out = c.backward(wants)
    for q in "xwb":
        if q not in wants:
            untouched = 7.0 if q == "b" else SENT
            assert bool((out[q] == untouched).all())
    Case([3, 150, 0, 40], 72, 40, act).check_backward(wants, num_rows=0)


def test_backward_against_differences():
    # the 64-bit loss <grad_y, y> along random directions of x, w and bias
    # (central differences, step 1e-4: truncation below 1e-7 of the value here);
    # the gradients' roundings are half a step of bf16 each, at random: four
    # standard deviations of their sum
    c = Case([7, 0, 30], 24, 16, "silu_glu", residual=False)
    y, z = c.forward(want_z=True)
    gy = bf16(c.rng.standard_normal((c.cap, c.N)))
    gy64 = gy.double().numpy()

    def loss(x, w, bias):
        t = 0.0
        for e, a, b in c.segments():
            t += (gy64[a:b] * R.act(x[a:b] @ w[e].T + bias[e], c.act, c.N)).sum()
        return t

    zt = bf16(np.nan_to_num(z))
    gx = torch.zeros((c.cap, c.K), dtype=torch.bfloat16, device="cuda")
    gw = torch.zeros((c.E, c.Nz, c.K), dtype=torch.bfloat16, device="cuda")
    gb = torch.zeros((c.E, c.Nz), device="cuda")
    ws = torch.zeros(M.mep_linear_workspace_bytes(c.cfg, c.cap), dtype=torch.uint8, device="cuda")
    M.mep_expert_linear_backward(c.cfg, c.dev(gy), c.dev(zt), c.dev(c.x), c.dev(c.w),
                                 c.dev(c.counts), c.dev(c.off), c.cap, 37, gx, gw, gb, ws)
    torch.cuda.synchronize()
    b64 = c.bias.astype(np.float64)
    h = 1e-4
    for seed in range(4):
        rng = np.random.default_rng(seed)
        dx, dw, db = (rng.standard_normal(s) for s in (c.x64.shape, c.w64.shape, b64.shape))
        dx[~c.used] = 0.0
        for args, got in (((dx, 0 * dw, 0 * db), gx), ((0 * dx, dw, 0 * db), gw),
                          ((0 * dx, 0 * dw, db), gb)):
            up = loss(c.x64 + h * args[0], c.w64 + h * args[1], b64 + h * args[2])
            dn = loss(c.x64 - h * args[0], c.w64 - h * args[1], b64 - h * args[2])
            num = (up - dn) / (2 * h)
            g = got.double().cpu().numpy()
            d = next(q for q in args if np.any(q))
            # z, grad_z and the gradient each round once: 3 half-steps of bf16
            noise = 4 * 3 * R.UBF16 * math.sqrt(((g * d) ** 2).sum())
            assert abs((g * d).sum() - num) <= noise + 1e-5 * abs(num), (seed, (g * d).sum(), num)


def test_offsets_past_32_bits():
    # the second segment's rows lie past 2^31 elements of em_x and grad_x
    K, N = 8192, 16
    rows = 2 ** 31 // K + 128
    counts = np.array([2, 3], np.int32)
    off = np.array([0, rows, rows + 128], np.int32)
    cap = rows + 128
    x = torch.zeros((cap, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x[rows:rows + 3] = torch.randn((3, K), generator=g, device="cuda").bfloat16()
    w = (torch.randn((2, N, K), generator=g, device="cuda") / 90).bfloat16()
    cfg = M.MepLinearConfig(2, K, N, M.MEP_ACT_NONE, M.MEP_QUANT_NONE)
    y = torch.zeros((cap, N), dtype=torch.bfloat16, device="cuda")
    ct, ot = torch.from_numpy(counts).cuda(), torch.from_numpy(off).cuda()
    M.mep_expert_linear(cfg, x, None, ct, ot, cap, 5, w, None, None, None, y, None)
    x3, w1 = x[rows:rows + 3].double().cpu().numpy(), w[1].double().cpu().numpy()
    ref, mag = x3 @ w1.T, np.abs(x3) @ np.abs(w1).T
    err = (K + 2) * R.U32 * mag
    assert np.all(np.abs(y[rows:rows + 3].double().cpu().numpy() - ref)
                  <= err + R.UBF16 * (np.abs(ref) + err))
    assert not bool(y[2:rows].any())
    gy = torch.zeros((cap, N), dtype=torch.bfloat16, device="cuda")
    gy[rows:rows + 3] = 1.0
    gx = torch.zeros((cap, K), dtype=torch.bfloat16, device="cuda")
    gw = torch.empty((2, N, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(M.mep_linear_workspace_bytes(cfg, cap), dtype=torch.uint8, device="cuda")
    M.mep_expert_linear_backward(cfg, gy, None, x, w, ct, ot, cap, 5, gx, gw, None, ws)
    sw, sx = w1.sum(0), x3.sum(0)
    got = gx[rows:rows + 3].double().cpu().numpy()
    assert np.all(np.abs(got - sw) <= 18 * R.U32 * np.abs(w1).sum(0) + 1.01 * R.UBF16 * np.abs(sw))
    got = gw[1].double().cpu().numpy()
    assert np.all(np.abs(got - sx) <= 5 * R.U32 * np.abs(x3).sum(0) + 1.01 * R.UBF16 * np.abs(sx))
    assert not bool(gw[0].any())


@pytest.mark.parametrize("act", list(ACT))
def test_segments_in_any_order(act):
    # the experts' segments do not ascend, and empty experts name any start
    c = Case([130, 0, 40, 7, 0, 300, 1, 0], 72, 40, act, extra=2)
    order = [5, 2, 7, 0, 3, 6, 1, 4]
    c.counts, starts = c.counts[order], c.off[:-1][order]
    starts[np.flatnonzero(c.counts == 0)] = [0, 384, 128]
    c.off = np.append(starts, c.off[-1]).astype(np.int32)
    c.check_forward(want_z=True)
    c.check_backward()


def test_segments_in_any_order_many_experts():
    counts = np.zeros(200, int)
    counts[[3, 64, 130, 199]] = 5, 200, 33, 129
    c = Case(counts, 24, 16, "silu_glu")
    order = np.random.default_rng(1).permutation(200)
    c.counts, c.off = c.counts[order], np.append(c.off[:-1][order], c.off[-1]).astype(np.int32)
    c.check_forward(num_rows=367)
    c.check_backward(num_rows=367)
