"""A mixture-of-experts block run as a model would: the norm before it (rows for the router,
rows or E4M3 codes for the dispatch), the grouped router, dispatch, experts and combine, the
norm, gate and residual after it, their gradients, and the clipping of all of them; from
bf16 and from FP8 dispatches, as HIP-graph replays and on several streams."""

import math

import numpy as np
import pytest
import torch

import combine_mep_plan_amd as M

import _block_ref as B
import _experts_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-6


def norm_cfg(H, post, pre, gate):
    return M.MepNormConfig(H, M.MEP_BF16, post, pre, gate, 1, EPS, 0.0, 1.0, 1.0)


class Block:
    """Buffers and weights: E experts over R ranks (a group each, `top` of which a token may
    use), hidden H, expert width I (gated), top-k of T tokens."""

    def __init__(self, T, H, I, ranks, epr, k, top, fp8=False, seed=0):
        self.T, self.H, self.I, self.k, self.E, self.fp8 = T, H, I, k, ranks * epr, fp8
        self.ranks, self.epr, self.top = ranks, epr, top
        E = self.E
        self.cap = T * k + 127 * E
        self.gate = M.MepGateConfig(E, k, M.MEP_SCORE_SIGMOID, M.MEP_BF16, 1, 2.0, 0.05)
        self.m = M.Mep(H, epr, k, T, ranks, quant=M.MEP_QUANT_FP8_CARRY if fp8 else M.MEP_QUANT_NONE,
                       scale_dim=H // 128 if fp8 else 0)
        q = M.MEP_QUANT_FP8_E4M3_BLOCK128 if fp8 else M.MEP_QUANT_NONE
        self.up = M.MepLinearConfig(E, H, I, M.MEP_ACT_SILU_GLU, q)
        self.down = M.MepLinearConfig(E, I, H, M.MEP_ACT_NONE, M.MEP_QUANT_NONE)
        self.router = M.MepLinearConfig(1, H, E, M.MEP_ACT_NONE, M.MEP_QUANT_NONE)
        self.before = norm_cfg(H, M.MEP_NORM_NONE, M.MEP_NORM_RMS, M.MEP_BLOCK_GATE_NONE)
        self.after = norm_cfg(H, M.MEP_NORM_RMS, M.MEP_NORM_RMS, M.MEP_BLOCK_GATE_TOKEN)
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, by=1.0: torch.randn(s, generator=g) * by  # noqa: E731
        w1 = n(E, 2 * I, H, by=1 / math.sqrt(H))
        self.w1s = None
        if fp8:
            s = torch.rand((E, 2 * I // 128, H // 128), generator=g) * 0.01 + 0.005
            blocks = s.repeat_interleave(128, 1).repeat_interleave(128, 2)
            self.w1, self.w1s = (w1 / blocks).clamp(-448, 448).to(torch.float8_e4m3fn).cuda(), s.cuda()
            self.w1_64 = self.w1.cpu().double() * blocks.double()
        else:
            self.w1 = w1.bfloat16().cuda()
            self.w1_64 = self.w1.cpu().double()
        self.w2 = n(E, H, I, by=1 / math.sqrt(I)).bfloat16().cuda()
        self.wr = n(1, E, H, by=1 / math.sqrt(H)).bfloat16().cuda()
        self.bias = n(E, by=0.1).cuda()
        self.w_in, self.w_post, self.w_next = ((1 + n(H, by=0.1)).cuda() for _ in range(3))
        z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
        bf, i32 = torch.bfloat16, torch.int32
        self.x, self.open = z(T, H, d=bf), z(T)
        self.n, self.logits = z(T, H, d=bf), z(T, E, d=bf)
        self.codes = z(T, H, d=torch.float8_e4m3fn) if fp8 else None
        self.scales = z(T, H // 128) if fp8 else None
        self.all_rows, self.one_segment = torch.tensor([T], dtype=i32, device="cuda"), z(2, d=i32)
        self.idx, self.w = z(T, k, d=i32), z(T, k)
        self.em_x = z(self.cap, H, d=torch.uint8 if fp8 else bf)
        self.em_s = z(self.cap, H // 128) if fp8 else None
        self.counts, self.off, self.src = z(E, d=i32), z(E + 1, d=i32), z(self.cap, d=i32)
        self.z1, self.h = z(self.cap, 2 * I, d=bf), z(self.cap, I, d=bf)
        self.y, self.out = z(self.cap, H, d=bf), z(T, H, d=bf)
        self.s, self.next, self.row = z(T, H, d=bf), z(T, H, d=bf), z(T, k, d=i32)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.x.copy_((torch.randn((self.T, self.H), generator=g) * 2).bfloat16())
        self.open.copy_(torch.randn(self.T, generator=g))

    def forward(self):
        T = self.T
        M.mep_block_norm(self.before, self.x, None, None, None, None, self.w_in, None, T, None, self.n,
                         self.codes, self.scales)
        M.mep_expert_linear(self.router, self.n, None, self.all_rows, self.one_segment, T, T, self.wr,
                            None, None, None, self.logits, None)
        M.mep_gate_grouped(self.gate, self.ranks, self.top, M.MEP_GROUP_TOP2, self.logits, self.bias, T,
                           self.idx, self.w)
        M.mep_dispatch_standard_moe(self.m.h, self.idx, T, self.codes if self.fp8 else self.n,
                                    self.scales, self.em_x, self.em_s, self.counts, self.off, self.src,
                                    self.cap)
        M.mep_expert_linear(self.up, self.em_x, self.em_s, self.counts, self.off, self.cap, T * self.k,
                            self.w1, self.w1s, None, None, self.h, self.z1)
        M.mep_expert_linear(self.down, self.h, None, self.counts, self.off, self.cap, T * self.k,
                            self.w2, None, None, None, self.y, None)
        M.mep_combine(self.m.h, M.MEP_EXPERT_MAJOR, self.y, self.w, self.out)
        M.mep_block_norm(self.after, self.x, self.out, self.open, self.w_post, None, self.w_next, None,
                         T, self.s, self.next, None, None)


def h64(t):
    return t.detach().cpu().double()


def rms(u, w):
    return u / torch.sqrt((u * u).mean(1, keepdim=True) + EPS) * w


def model(L, x, open_, w_in, wr, w1, w2, w_post, w_next, rows=None):
    """(stream, next rows, balance-free output) of the definitions in 64 bits, for the experts
    that the device chose.  rows: what the experts read, where it is not the norm's result."""
    idx = L.idx.cpu().long()
    n = rms(x, w_in)
    v = torch.sigmoid(n @ wr[0].T).gather(1, idx)
    w = 2.0 * v / v.sum(1, keepdim=True)
    read = n if rows is None else rows
    out = torch.zeros_like(x)
    for e in range(L.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            z = read[t] @ w1[e].T
            y = (torch.nn.functional.silu(z[:, :L.I]) * z[:, L.I:]) @ w2[e].T
            out = out.index_add(0, t, w[t, j][:, None] * y)
    s = x + torch.sigmoid(open_)[:, None] * rms(out, w_post)
    return s, rms(s, w_next)


@pytest.mark.parametrize("T,H,I,ranks,epr,k,top,fp8", [
    (1, 256, 128, 4, 4, 3, 2, False), (130, 512, 128, 8, 4, 6, 3, False), (301, 264, 72, 4, 2, 2, 1, False),
    (1, 256, 128, 4, 4, 3, 2, True), (333, 512, 256, 8, 4, 8, 4, True)])
def test_forward(T, H, I, ranks, epr, k, top, fp8):
    L = Block(T, H, I, ranks, epr, k, top, fp8)
    L.fill(T)
    L.forward()
    torch.cuda.synchronize()
    assert M.mep_get_status(L.m.h) == 0
    idx = L.idx.cpu().numpy()
    logits = h64(L.logits).numpy()
    ridx, rw = B.grouped(logits, h64(L.bias).numpy(), k, "sigmoid", 1, 2.0, ranks, top, "top2")
    assert np.array_equal(idx, ridx)
    assert np.all(np.abs(h64(L.w).numpy() - rw) <= R.prob_steps() * R.U32 * rw)
    assert all(len(set(row // epr)) <= top for row in idx)  # ranks a token goes to
    rows = None
    if fp8:
        M.mep_get_route(L.m.h, None, L.row)
        at = L.row[:, 0].long()
        codes = h64(L.em_x.view(torch.float8_e4m3fn)[at])
        rows = codes * h64(L.em_s[at]).repeat_interleave(128, 1)
        # what the dispatch carried is the norm's codes
        assert torch.equal(L.em_x[at].cpu(), L.codes.view(torch.uint8).cpu())
        n64 = rms(h64(L.x), h64(L.w_in))
        assert float((rows - n64).norm() / n64.norm()) <= 2.0 ** -4
    s, nxt = model(L, *(h64(t) for t in (L.x, L.open, L.w_in, L.wr)), L.w1_64, h64(L.w2),
                   h64(L.w_post), h64(L.w_next), rows)
    # n, logits, h, y and out each round to bf16 once on the way, s and next once more, with
    # independent signs; a logit's rounding moves a sigmoid by less than its own size, and
    # the norm after the block keeps relative errors: below 8 half-steps of the norm
    for got, ref in ((L.s, s), (L.next, nxt)):
        off = (h64(got) - ref).norm() / ref.norm()
        assert off <= 8 * R.UBF16, float(off)


class Training(Block):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        z = torch.zeros_like
        self.gs, self.gnext = z(self.s), z(self.next)
        self.gx, self.gout, self.gopen = z(self.x), z(self.out), z(self.open)
        self.gy, self.gh, self.gem = z(self.y), z(self.h), z(self.em_x)
        self.gw, self.glogits, self.gn, self.gin = z(self.w), z(self.logits), z(self.n), z(self.x)
        self.bal = (torch.zeros(self.E + 1, dtype=torch.int32, device="cuda"),
                    torch.zeros(self.E, device="cuda"), torch.zeros(1, device="cuda"))
        self.weights = ("w1", "w2", "wr", "w_in", "w_post", "w_next")
        self.grads = [z(getattr(self, n)) for n in self.weights]
        self.clipped = [z(g) for g in self.grads]
        self.list, self.norm = M.MepGrads(self.grads, self.clipped), torch.zeros(1, device="cuda")
        ws = max([M.mep_linear_workspace_bytes(c, self.cap) for c in (self.up, self.down, self.router)]
                 + [M.mep_block_norm_workspace_bytes(c, self.T) for c in (self.before, self.after)]
                 + [M.mep_grad_workspace_bytes(self.list)])
        self.ws = torch.zeros(ws, dtype=torch.uint8, device="cuda")

    def fill(self, seed):
        super().fill(seed)
        g = torch.Generator().manual_seed(seed + 1000)
        for t in (self.gs, self.gnext):
            t.copy_(torch.randn((self.T, self.H), generator=g).bfloat16())

    def backward(self, limit=1.0):
        T, ws = self.T, self.ws
        gw1, gw2, gwr, gw_in, gw_post, gw_next = self.grads
        M.mep_block_norm_backward(self.after, self.gs, self.gnext, self.s, self.out, self.open,
                                  self.w_post, None, self.w_next, T, self.gx, self.gout, self.gopen,
                                  gw_post, None, gw_next, None, ws)
        # the combine's own gradient is two lines of torch: the rows' and the weights'
        M.mep_get_route(self.m.h, None, self.row)
        rows = self.row.long()
        self.gy.zero_()
        self.gy[rows.reshape(-1)] = (self.w[..., None] * self.gout[:, None].float()).to(
            torch.bfloat16).reshape(-1, self.H)
        self.gw.copy_((self.gout[:, None].float() * self.y[rows].float()).sum(-1))
        M.mep_expert_linear_backward(self.down, self.gy, None, self.h, self.w2, self.counts, self.off,
                                     self.cap, T * self.k, self.gh, gw2, None, ws)
        M.mep_expert_linear_backward(self.up, self.gh, self.z1, self.em_x, self.w1, self.counts,
                                     self.off, self.cap, T * self.k, self.gem, gw1, None, ws)
        M.mep_gate_backward(self.gate, self.logits, self.idx, None, T, self.gw, None, None, self.glogits)
        M.mep_expert_linear_backward(self.router, self.glogits, None, self.n, self.wr, self.all_rows,
                                     self.one_segment, T, T, self.gn, gwr, None, ws)
        self.gn.copy_(self.gn.float() + self.gem[rows].float().sum(1))
        M.mep_block_norm_backward(self.before, self.gx, self.gn, self.x, None, None, None, None,
                                  self.w_in, T, self.gin, None, None, None, None, gw_in, None, ws)
        M.mep_grad_norm(self.list, self.norm, ws)
        M.mep_grad_clip(self.list, self.norm, limit)

    def results(self):
        return [self.idx, self.w, self.s, self.next, self.gin, self.gopen, *self.grads, self.norm,
                *self.clipped]


def test_training_step():
    L = Training(90, 128, 64, 4, 4, 3, 2)
    L.fill(3)
    L.forward()
    L.backward(0.5)
    torch.cuda.synchronize()
    leaves = [h64(t).requires_grad_(True) for t in (L.x, L.open, L.w_in, L.wr, L.w1, L.w2, L.w_post,
                                                    L.w_next)]
    s, nxt = model(L, *leaves)
    total = (s * h64(L.gs)).sum() + (nxt * h64(L.gnext)).sum()
    want = dict(zip(("x", "open", "w_in", "wr", "w1", "w2", "w_post", "w_next"),
                    torch.autograd.grad(total, leaves)))
    got = dict(zip(L.weights, L.grads), x=L.gin, open=L.gopen)
    # Each gradient is a sum of many terms, each with at most 14 roundings to bf16 on its
    # way (n, logits, z, h, y, out, s and the gradients of s, out, y, h, z, n and the
    # results) of independent signs: relative to its norm below 14 half-steps of bf16.
    for n, ref in want.items():
        off = (h64(got[n]) - ref).norm() / ref.norm()
        assert off <= 14 * R.UBF16, (n, float(off))
    norm = math.sqrt(sum(float(h64(g).square().sum()) for g in L.grads))
    assert abs(float(L.norm) - norm) <= 1.01 * R.U32 * norm
    for g, c in zip(L.grads, L.clipped):
        u = R.UBF16 if g.dtype == torch.bfloat16 else R.U32
        ref = h64(g) * min(1.0, 0.5 / (norm + 1e-6))
        assert bool(((h64(c) - ref).abs() <= (u + 4 * R.U32) * ref.abs() + 1e-45).all())


def test_graph_replays_give_the_eager_results():
    L = Training(200, 256, 128, 4, 4, 4, 2)
    eager = {}
    for seed in (1, 2, 3):
        L.fill(seed)
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
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(L.results(), eager[seed]):
            assert torch.equal(a, b)
        # the program's own eager work between replays, on the same workspaces
        L.fill(7)
        L.forward()
        L.backward()
        torch.cuda.synchronize()


def test_two_graphs_share_a_workspace():
    # captured apart, replayed in turn: nothing of one stays in the workspace for the other
    L = Training(150, 256, 128, 4, 4, 4, 2)
    L.fill(5)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in L.results()]
    graphs = []
    for limit in (1.0, 1e6):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.forward()
            L.backward(limit)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        got = L.results()
        n = len(L.clipped)
        assert all(torch.equal(a, b) for a, b in zip(got[:-n], want[:-n]))
        assert all(torch.equal(a, b) for a, b in zip(L.clipped, want[-n:] if i == 0 else L.grads))


def test_blocks_on_two_streams_at_once():
    blocks = [Training(300, 256, 128, 4, 4, 4, 2, seed=s) for s in (0, 1)]
    want = []
    for i, L in enumerate(blocks):
        L.fill(10 + i)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.results()])
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(4):
        for L, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                L.forward()
                L.backward()
    torch.cuda.synchronize()
    for L, w in zip(blocks, want):
        assert all(torch.equal(a, b) for a, b in zip(L.results(), w))
