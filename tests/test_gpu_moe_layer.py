"""Router, dispatch, experts and combine run together as a layer would: forward
from bf16 and from FP8 dispatches, a training step with the gradients, HIP-graph
replays and calls on several streams."""

import math

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _experts_ref as R

pytestmark = pytest.mark.gpu


class Layer:
    """Buffers and weights of one MoE layer: E experts over R ranks, hidden H, expert
    width I (gated), top-k of T tokens."""

    def __init__(self, T, H, I, ranks, epr, k, fp8=False, score="sigmoid", seed=0):
        self.T, self.H, self.I, self.k, self.E, self.fp8 = T, H, I, k, ranks * epr, fp8
        E = self.E
        self.cap = T * k + 127 * E
        sigmoid = score == "sigmoid"
        self.score = score
        self.gate = M.MepGateConfig(E, k, M.MEP_SCORE_SIGMOID if sigmoid else M.MEP_SCORE_SOFTMAX,
                                    M.MEP_FP32, 1, 1.5, 0.05)
        self.m = M.Mep(H, epr, k, T, ranks, fp8=fp8)
        q = M.MEP_QUANT_FP8_E4M3_BLOCK128 if fp8 else M.MEP_QUANT_NONE
        self.up = M.MepLinearConfig(E, H, I, M.MEP_ACT_SILU_GLU, q)
        self.down = M.MepLinearConfig(E, I, H, M.MEP_ACT_NONE, M.MEP_QUANT_NONE)
        g = torch.Generator().manual_seed(seed)
        w1 = torch.randn((E, 2 * I, H), generator=g) / math.sqrt(H)
        w2 = torch.randn((E, H, I), generator=g) / math.sqrt(I)
        self.bias = torch.randn(E, generator=g).mul(0.1).cuda() if sigmoid else None
        self.w1s = None
        if fp8:
            s = torch.rand((E, 2 * I // 128, H // 128), generator=g) * 0.01 + 0.005
            blocks = s.repeat_interleave(128, 1).repeat_interleave(128, 2)
            self.w1 = (w1 / blocks).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
            self.w1s = s.cuda()
            self.w1_64 = self.w1.cpu().double() * blocks.double()
        else:
            self.w1 = w1.bfloat16().cuda()
            self.w1_64 = self.w1.cpu().double()
        self.w2 = w2.bfloat16().cuda()
        z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.logits, self.x = z(T, E), z(T, H, d=bf)
        self.idx, self.w = z(T, k, d=torch.int32), z(T, k)
        self.em_x = z(self.cap, H, d=torch.uint8 if fp8 else bf)
        self.em_s = z(self.cap, H // 128) if fp8 else None
        self.counts, self.off = z(E, d=torch.int32), z(E + 1, d=torch.int32)
        self.src = z(self.cap, d=torch.int32)
        self.z1, self.h = z(self.cap, 2 * I, d=bf), z(self.cap, I, d=bf)
        self.y, self.out = z(self.cap, H, d=bf), z(T, H, d=bf)
        self.row = z(T, k, d=torch.int32)
        self.bal = (z(E + 1, d=torch.int32), z(E), z(1))
        self.bal_ws = torch.zeros(M.mep_balance_workspace_bytes(self.gate, T), dtype=torch.uint8,
                                  device="cuda")

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.logits.copy_(torch.randn((self.T, self.E), generator=g))
        self.x.copy_(torch.randn((self.T, self.H), generator=g).bfloat16())

    def forward(self, stream=None):
        T = self.T
        M.mep_gate(self.gate, self.logits, self.bias, T, self.idx, self.w, stream)
        M.mep_balance_loss(self.gate, self.logits, self.idx, None, T, *self.bal, self.bal_ws,
                           stream)
        M.mep_dispatch_standard_moe(self.m.h, self.idx, T, self.x, None, self.em_x, self.em_s,
                                    self.counts, self.off, self.src, self.cap, stream)
        M.mep_expert_linear(self.up, self.em_x, self.em_s, self.counts, self.off, self.cap,
                            T * self.k, self.w1, self.w1s, None, None, self.h, self.z1, stream)
        M.mep_expert_linear(self.down, self.h, None, self.counts, self.off, self.cap, T * self.k,
                            self.w2, None, None, None, self.y, None, stream)
        M.mep_combine(self.m.h, M.MEP_EXPERT_MAJOR, self.y, self.w, self.out, stream)

    def host(self, t):
        return t.cpu().double().numpy()


def reference(L, x64):
    """(output, bound) of the layer for the routing on the device: h and y round to
    bf16 once each, the output once, sums in fp32."""
    idx, w = L.idx.cpu().numpy(), L.host(L.w)
    w1, w2 = L.w1_64.numpy(), L.host(L.w2)
    out, err = np.zeros((L.T, L.H)), np.zeros((L.T, L.H))
    for e in range(L.E):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        z = x64[t] @ w1[e].T
        dz = (L.H + 2) * R.U32 * (np.abs(x64[t]) @ np.abs(w1[e]).T)
        g, u = z[:, : L.I], z[:, L.I:]
        h = R.act(z, "silu_glu", L.I)
        s = np.abs(R.act(g, "silu", L.I))
        dg, du = dz[:, : L.I], dz[:, L.I:]
        dh = 1.13 * dg * (np.abs(u) + du) + (s + 1.13 * dg) * du + 8 * R.U32 * np.abs(h)
        dh = dh + R.UBF16 * (np.abs(h) + dh)
        y = h @ w2[e].T
        dy = dh @ np.abs(w2[e]).T + (L.I + 2) * R.U32 * ((np.abs(h) + dh) @ np.abs(w2[e]).T)
        dy = dy + R.UBF16 * (np.abs(y) + dy)
        np.add.at(out, t, w[t, j][:, None] * y)
        np.add.at(err, t, np.abs(w[t, j])[:, None] * dy + (L.k + 1) * R.U32 * np.abs(
            w[t, j][:, None] * y))
    return out, err + R.UBF16 * (np.abs(out) + err)


@pytest.mark.parametrize("T,H,I,ranks,epr,k,fp8,score", [
    (1, 256, 128, 4, 2, 2, False, "softmax"), (130, 512, 256, 8, 4, 8, False, "sigmoid"),
    (700, 264, 72, 2, 3, 3, False, "softmax"), (1, 256, 128, 4, 2, 2, True, "sigmoid"),
    (333, 512, 256, 8, 2, 6, True, "softmax")])
def test_forward(T, H, I, ranks, epr, k, fp8, score):
    L = Layer(T, H, I, ranks, epr, k, fp8, score)
    L.fill(T)
    L.forward()
    torch.cuda.synchronize()
    assert M.mep_get_status(L.m.h) == 0
    idx = L.idx.cpu().numpy()
    logits = L.host(L.logits)
    bias = None if L.bias is None else L.host(L.bias)
    ridx, rw = R.gate(logits, bias, k, score, 1, 1.5)
    assert np.array_equal(idx, ridx)
    assert np.all(np.abs(L.host(L.w) - rw) <= R.prob_steps() * R.U32 * rw)
    # the dispatch and the balance loss count the same experts
    assert np.array_equal(L.counts.cpu().numpy(), np.bincount(idx.reshape(-1), minlength=L.E))
    assert np.array_equal(L.bal[0].cpu().numpy(), np.append(L.counts.cpu().numpy(), T))
    x64 = L.host(L.x)
    if fp8:  # what the dispatch's codes and scales stand for
        M.mep_get_route(L.m.h, None, L.row)
        rows = L.row.cpu().numpy()[:, 0]
        codes = L.em_x.cpu().view(torch.float8_e4m3fn).double().numpy()[rows]
        x64 = codes * np.repeat(L.host(L.em_s)[rows], 128, axis=1)
    ref, err = reference(L, x64)
    assert np.all(np.abs(L.host(L.out) - ref) <= err)


class Training(Layer):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        z = torch.zeros_like
        self.gout, self.gw, self.gl = z(self.out), z(self.w), torch.ones(1, device="cuda")
        self.gy, self.gh, self.gx = z(self.y), z(self.h), z(self.em_x)
        self.gw1, self.gw2, self.glogits = z(self.w1), z(self.w2), z(self.logits)
        n = max(M.mep_linear_workspace_bytes(c, self.cap) for c in (self.up, self.down))
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def backward(self, stream=None):
        """The combine's own gradient is two lines of torch: the rows' and the weights'."""
        M.mep_get_route(self.m.h, None, self.row, stream)
        rows = self.row.long()
        self.gy.zero_()
        self.gy[rows.reshape(-1)] = (self.w[..., None] * self.gout[:, None].float()).to(
            torch.bfloat16).reshape(-1, self.H)
        self.gw.copy_((self.gout[:, None].float() * self.y[rows].float()).sum(-1))
        M.mep_expert_linear_backward(self.down, self.gy, None, self.h, self.w2, self.counts,
                                     self.off, self.cap, self.T * self.k, self.gh, self.gw2, None,
                                     self.ws, stream)
        M.mep_expert_linear_backward(self.up, self.gh, self.z1, self.em_x, self.w1, self.counts,
                                     self.off, self.cap, self.T * self.k, self.gx, self.gw1, None,
                                     self.ws, stream)
        M.mep_gate_backward(self.gate, self.logits, self.idx, None, self.T, self.gw, self.bal[0],
                            self.gl, self.glogits, stream)

    def results(self):
        # of grad_x the routed rows: the others are not written
        return [self.idx, self.w, self.out, *self.bal, self.gw1, self.gw2, self.glogits,
                self.gx[self.row.long()]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step(score):
    T, H, I, k = 90, 128, 64, 4
    L = Training(T, H, I, 4, 3, k, score=score)
    L.fill(3)
    L.gout.copy_(torch.randn((T, H), generator=torch.Generator().manual_seed(9)).bfloat16())
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    # the same loss by 64-bit autograd, on the device's routing
    idx = L.idx.cpu().long()
    logits, w1, w2 = (t.cpu().double().requires_grad_(True) for t in (L.logits, L.w1, L.w2))
    x = L.x.cpu().double()
    v = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    p = v / v.sum(1, keepdim=True)
    w = v.gather(1, idx)
    w = 1.5 * w / w.sum(1, keepdim=True)
    z = torch.einsum("th,tjnh->tjn", x, w1[idx])
    h = torch.nn.functional.silu(z[..., :I]) * z[..., I:]
    y = torch.einsum("tji,tjhi->tjh", h, w2[idx])
    out = (w[..., None] * y).sum(1)
    counts = torch.bincount(idx.reshape(-1), minlength=L.E).double()
    loss = 0.05 * L.E / (k * T) * (counts * p.mean(0)).sum()
    want = float(loss.detach())
    assert abs(float(L.bal[2]) - want) <= 300 * R.U32 * want
    total = (out * L.gout.cpu().double()).sum() + loss
    grads = torch.autograd.grad(total, (logits, w1, w2))
    # Each gradient is a sum of many terms, each with at most 8 roundings to bf16
    # on its way (h, z, y, grad_y, grad_h, grad_z and the results) of independent
    # signs: relative to its norm the error is below 8 half-steps of bf16.
    for got, ref in zip((L.glogits, L.gw1, L.gw2), grads):
        off = (got.cpu().double() - ref).norm() / ref.norm()
        assert off <= 8 * R.UBF16, off


def test_graph_replays_give_the_eager_results():
    L = Training(200, 256, 128, 4, 4, 4)
    eager = {}
    for seed in (1, 2, 3):
        L.fill(seed)
        L.gout.copy_(L.x)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        eager[seed] = [t.clone() for t in L.results()]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        L.forward()
        L.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward()
        L.backward()
    for seed in (2, 1, 3, 3, 2):
        L.fill(seed)
        L.gout.copy_(L.x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(L.results(), eager[seed]):
            assert torch.equal(a, b)
        # the program's own eager work between replays, on the same workspaces
        L.fill(7)
        L.forward()
        torch.cuda.synchronize()


def test_layers_on_two_streams_at_once():
    layers = [Training(300, 256, 128, 4, 4, 4, seed=s) for s in (0, 1)]
    want = []
    for i, L in enumerate(layers):
        L.fill(10 + i)
        L.gout.copy_(L.x)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.results()])
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(4):
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.forward()
                L.backward()
    torch.cuda.synchronize()
    assert len(layers) == len(want)
    for L, w in zip(layers, want):
        for a, b in zip(L.results(), w):
            assert torch.equal(a, b)
