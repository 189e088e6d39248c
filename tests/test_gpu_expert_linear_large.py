"""The experts' product and its gradients in tiles of 256 x 256, which the sizes of
``test_gpu_expert_linear`` do not reach: each case first works out the launch's
rule, so that it says so if it no longer takes these tiles.  Bounds as there, and
for whole segments the norm of the error: a rounding to bf16 is off by a uniform
share of half a step, 2^-8 of a value at most, so all together by 2^-8 / sqrt(3) of
the norm, beside which the accumulation's part vanishes."""

import math

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _experts_ref as R
from test_gpu_expert_linear import ACT, Case

pytestmark = pytest.mark.gpu

# whole row tiles with a rest behind them (from four on, out of order), one row
# more than a tile, no row, few rows
COUNTS = [1100, 0, 1300, 257, 40]


def takes_large_tiles(cols, cols_a_tile, rows, E):
    used = min(rows, E)
    return -(-cols // cols_a_tile) * (rows // 256 + used) >= 144 and rows > 64 * used


class Large(Case):
    def lost_in_groups(self, e, a, b):
        x = torch.from_numpy(np.abs(self.x64[a:b])).cuda()
        w = torch.from_numpy(np.abs(self.w64[e])).cuda()
        lost = torch.zeros((b - a, self.Nz), dtype=torch.float64, device="cuda")
        for k in range(0, self.K, 8):
            largest = x[:, k, None] * w[None, :, k]
            for q in range(k + 1, k + 8):
                torch.maximum(largest, x[:, q, None] * w[None, :, q], out=largest)
            lost += 7 * 2.0 ** -13 * largest
        return lost.cpu().numpy()

    def check_large_forward(self):
        rows = int(self.counts.sum())
        assert takes_large_tiles(self.N, 128 if self.act == "silu_glu" else 256, rows, self.E)
        self.check_forward(want_z=True)
        if not self.fp8:
            _, z = self.forward(want_z=True)
            for e, a, b in self.segments():
                ref = self.x64[a:b] @ self.w64[e].T
                if self.bias is not None:
                    ref += self.bias[e]
                off = np.linalg.norm(z[a:b] - ref) / np.linalg.norm(ref)
                assert off <= R.UBF16 / math.sqrt(3), off

    def check_large_backward(self, x=True, w=True):
        rows = int(self.counts.sum())
        if x:
            assert takes_large_tiles(self.K, 256, rows, self.E)
        if w:
            assert self.E * -(-self.Nz // 256) * -(-self.K // 256) >= 144
        self.check_backward()


def columns(act):
    return 1240 if act == "silu_glu" else 2504  # the last column tile is in part


@pytest.mark.parametrize("act", list(ACT))
def test_forward(act):
    Large(COUNTS, 192, columns(act), act, extra=5).check_large_forward()


@pytest.mark.parametrize("act", ["none", "silu_glu"])
@pytest.mark.parametrize("K", [8, 64, 72, 128, 200, 256, 320])
def test_forward_depths(K, act):
    # no, one and more steps, odd and even, with and without a rest
    Large(COUNTS, K, columns(act), act, extra=5).check_large_forward()


@pytest.mark.parametrize("act", list(ACT))
def test_forward_fp8(act):
    N = 1280 if act == "silu_glu" else 2432
    Large(COUNTS, 256, N, act, fp8=True, extra=5).check_large_forward()


@pytest.mark.parametrize("act", ["none", "silu_glu"])
@pytest.mark.parametrize("K", [128, 384, 512, 640])
def test_forward_depths_fp8(K, act):
    N = 1280 if act == "silu_glu" else 2432
    Large(COUNTS, K, N, act, bias=False, residual=False, fp8=True).check_large_forward()


@pytest.mark.parametrize("fp8", [False, True])
def test_forward_of_a_deep_product(fp8):
    Large([700, 300, 450], 7168, 2304, "silu_glu", bias=False, residual=False,
          fp8=fp8).check_large_forward()


def test_rows_past_the_capacity():
    c = Large(COUNTS, 136, 2504, "silu", cap=1152 + 1200)
    c.check_large_forward()
    c.check_backward()


@pytest.mark.parametrize("Nz", [8, 64, 72, 128, 192, 200, 256, 320])
def test_backward_depths(Nz):
    # grad_x sums over Nz: no, one and more steps, odd and even, with and without a rest
    Large(COUNTS, 2504, Nz, "none", extra=5).check_large_backward(w=False)


@pytest.mark.parametrize("act", list(ACT))
def test_backward(act):
    Large(COUNTS, 2504, 264 if act == "silu_glu" else 520, act,
          extra=5).check_large_backward()


@pytest.mark.parametrize("fp8", [False, True])
def test_most_experts_in_large_tiles(fp8):
    # 4096 experts' row tiles beside the operands in LDS
    E, n, K, N = 4096, 65, 128, 128
    rows, cap = E * n, E * 128
    assert takes_large_tiles(N, 256, rows, E) and takes_large_tiles(K, 256, rows, E)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t = torch.float8_e4m3fn if fp8 else torch.bfloat16
    x, w = normal(E, 128, K).to(t), normal(E, N, K).to(t)
    ct = torch.full((E,), n, dtype=torch.int32, device="cuda")
    ot = torch.arange(0, cap + 1, 128, dtype=torch.int32, device="cuda")
    one = lambda *s: torch.ones(s, device="cuda") if fp8 else None  # noqa: E731
    cfg = M.MepLinearConfig(E, K, N, M.MEP_ACT_NONE, M.MEP_QUANT_FP8_E4M3_BLOCK128 if fp8
                            else M.MEP_QUANT_NONE)
    y = torch.full((E, 128, N), 7.0, dtype=torch.bfloat16, device="cuda")
    M.mep_expert_linear(cfg, x, one(cap, 1), ct, ot, cap, rows, w, one(E, 1, 1), None, None, y,
                        None)
    x64, wt = x[:, :n].double(), w.double().transpose(1, 2).contiguous()
    ref, mag = torch.matmul(x64, wt), torch.matmul(x64.abs(), wt.abs())
    # E4M3: 7 * 2^-13 of the largest product in each group of 8, so of the magnitudes
    err = (K + 2) * R.U32 * mag + (7 * 2.0 ** -13 * mag if fp8 else 0.0)
    assert bool(((y[:, :n].double() - ref).abs() <= err + R.UBF16 * (ref.abs() + err)).all())
    assert bool((y[:, n:] == 7.0).all())
    if fp8:
        return
    gx = torch.full((E, 128, K), 7.0, dtype=torch.bfloat16, device="cuda")
    gy = normal(E, 128, N).bfloat16()
    ws = torch.empty(M.mep_linear_workspace_bytes(cfg, cap), dtype=torch.uint8, device="cuda")
    M.mep_expert_linear_backward(cfg, gy, None, x, w, ct, ot, cap, rows, gx, None, None, ws)
    g64, w64 = gy[:, :n].double(), w.double()
    ref = torch.matmul(g64, w64)
    err = (N + 2) * R.U32 * torch.matmul(g64.abs(), w64.abs())
    assert bool(((gx[:, :n].double() - ref).abs() <= err + R.UBF16 * (ref.abs() + err)).all())
    assert bool((gx[:, n:] == 7.0).all())


def test_offsets_past_32_bits():
    # the second segment lies past 2^31 elements of x, y and their gradients
    K, N, rows = 9160, 9104, 640
    first = (2 ** 31 // N // 128 + 1) * 128
    cap = first + rows
    assert first * min(K, N) > 2 ** 31
    assert takes_large_tiles(N, 256, rows + 2, 2) and takes_large_tiles(K, 256, rows + 2, 2)
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    new = lambda r, c: torch.zeros((r, c), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, gy, y, gx = new(cap, K), new(cap, N), new(cap, N), new(cap, K)
    x[first:] = normal(rows, K).bfloat16()
    gy[first:] = normal(rows, N).bfloat16()
    w = (normal(2, N, K) / 96).bfloat16()
    gw = torch.empty((2, N, K), dtype=torch.bfloat16, device="cuda")
    ct = torch.tensor([2, rows], dtype=torch.int32, device="cuda")
    ot = torch.tensor([0, first, cap], dtype=torch.int32, device="cuda")
    cfg = M.MepLinearConfig(2, K, N, M.MEP_ACT_NONE, M.MEP_QUANT_NONE)
    M.mep_expert_linear(cfg, x, None, ct, ot, cap, rows + 2, w, None, None, None, y, None)
    ws = torch.empty(M.mep_linear_workspace_bytes(cfg, cap), dtype=torch.uint8, device="cuda")
    M.mep_expert_linear_backward(cfg, gy, None, x, w, ct, ot, cap, rows + 2, gx, gw, None, ws)
    x64, w64, g64 = x[first:].double(), w[1].double(), gy[first:].double()
    for got, a, b, steps in ((y[first:], x64, w64.T.contiguous(), K), (gx[first:], g64, w64, N),
                             (gw[1], g64.T.contiguous(), x64, rows)):
        ref, err = a @ b, (steps + 2) * R.U32 * (a.abs() @ b.abs())
        assert bool(((got.double() - ref).abs() <= err + R.UBF16 * (ref.abs() + err)).all())
        assert float((got.double() - ref).norm() / ref.norm()) <= R.UBF16 / math.sqrt(3)
    assert not bool(gw[0].any()) and not bool(y[:first].any()) and not bool(gx[:first].any())
    del x, gy, y, gx, w, gw, ws
    torch.cuda.empty_cache()
