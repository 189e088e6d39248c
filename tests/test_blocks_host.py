"""Host-side checks of the grouped router, the norms around a block and the calls over many
gradients (no GPU, nothing launched): configs, sizes, null pointers, alignment, workspaces,
and the binding's own checks of tensors.  Device pointers are fake aligned addresses."""

import ctypes as C

import pytest
import torch

import combine_mep_plan_amd as M

F = 0x7F0000000000  # never dereferenced on the host
NULL, CONFIG, SHAPE, ALIGN = M.MEP_ERR_NULL, M.MEP_ERR_CONFIG, M.MEP_ERR_SHAPE, M.MEP_ERR_ALIGN


def gate_cfg(**kw):
    base = dict(num_experts=256, top_k=8, score=M.MEP_SCORE_SOFTMAX, dtype=M.MEP_FP32, normalize=1,
                scale=1.0, balance_coef=0.0)
    return M.MepGateConfig(**{**base, **kw})


def grouped(c, groups=8, top=4, by=M.MEP_GROUP_TOP2, logits=F, bias=None, T=4, indices=F, weights=F):
    return M.lib().mep_gate_grouped(C.byref(c) if c else None, groups, top, by, logits, bias, T,
                                    indices, weights, None)


def norm_cfg(**kw):
    base = dict(hidden_dim=7168, dtype=M.MEP_BF16, post=M.MEP_NORM_RMS, pre=M.MEP_NORM_RMS,
                gate=M.MEP_BLOCK_GATE_NONE, gate_sigmoid=0, eps=1e-6, weight_offset=0.0,
                residual_scale=1.0, block_scale=1.0)
    return M.MepNormConfig(**{**base, **kw})


def norm(c, x=F, y=F, gate=None, wp=F, bp=None, wn=F, bn=None, T=4, s=F, n=F, codes=None, scales=None):
    return M.lib().mep_block_norm(C.byref(c) if c else None, x, y, gate, wp, bp, wn, bn, T, s, n,
                                  codes, scales, None)


def backward(c, gs=F, gn=F, s=F, y=F, gate=None, wp=F, bp=None, wn=F, T=4, gx=F, gy=F, gg=None, gwp=F,
             gbp=None, gwn=F, gbn=None, ws=F, size=1 << 40):
    return M.lib().mep_block_norm_backward(C.byref(c) if c else None, gs, gn, s, y, gate, wp, bp, wn,
                                           T, gx, gy, gg, gwp, gbp, gwn, gbn, ws, size, None)


def grads(*rows):
    a = (M.MepGrad * max(1, len(rows)))()
    for i, (data, out, numel, dtype) in enumerate(rows):
        a[i] = M.MepGrad(data, out, numel, dtype, 0)
    return a, len(rows)


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=65), dict(groups=7), dict(groups=-8),
                                dict(top=0), dict(top=9), dict(by=2), dict(by=-1),
                                dict(groups=64, top=1)])
def test_bad_groups(kw):
    # 64 groups of 4 experts: one of them holds fewer than k
    assert grouped(gate_cfg(), **kw) == CONFIG


def test_grouped_refusals():
    c = gate_cfg()
    assert grouped(None) == NULL
    assert grouped(gate_cfg(top_k=0)) == grouped(gate_cfg(num_experts=4097)) == CONFIG
    assert grouped(gate_cfg(num_experts=8, top_k=2), 8, 2) == CONFIG  # the two best of one expert
    assert grouped(c, T=-1) == grouped(c, T=(1 << 26) + 1) == SHAPE
    for kw in (dict(logits=None), dict(indices=None), dict(weights=None)):
        assert grouped(c, **kw) == NULL
    for kw in (dict(logits=F + 4), dict(indices=F + 8), dict(weights=F + 4)):
        assert grouped(c, **kw) == ALIGN
    assert grouped(c, bias=F) == CONFIG  # a bias needs sigmoid scores
    assert grouped(gate_cfg(score=M.MEP_SCORE_SIGMOID), bias=F + 4) == ALIGN
    assert grouped(c, logits=None, indices=None, weights=None, T=0) == M.MEP_OK


@pytest.mark.parametrize("kw", [dict(hidden_dim=0), dict(hidden_dim=-8), dict(hidden_dim=12),
                                dict(hidden_dim=16392), dict(dtype=2), dict(post=3), dict(pre=-1),
                                dict(gate=3), dict(gate=-1), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(eps=float("inf"))])
def test_bad_norm_configs(kw):
    c = norm_cfg(**kw)
    assert norm(c) == backward(c) == CONFIG
    assert M.mep_block_norm_workspace_bytes(c, 4) == 0


def test_norm_refusals():
    c = norm_cfg()
    token = norm_cfg(gate=M.MEP_BLOCK_GATE_TOKEN)
    assert norm(None) == NULL
    assert norm(c, T=-1) == norm(c, T=(1 << 26) + 1) == SHAPE
    assert norm(c, x=None, y=None) == NULL
    assert norm(c, s=None, n=None) == NULL
    assert norm(token) == NULL                      # a gate is named and not given
    assert norm(c, gate=F) == CONFIG                # given and not named
    assert norm(token, y=None, gate=F) == NULL      # nothing to gate
    assert norm(c, codes=F) == norm(c, scales=F) == NULL
    assert norm(norm_cfg(hidden_dim=520), codes=F, scales=F) == CONFIG
    names = ("x", "y", "wp", "bp", "wn", "bn", "s", "n")
    for name in names:
        assert norm(c, **{name: F + 8}) == ALIGN, name
    assert norm(token, gate=F + 4) == norm(c, codes=F + 8, scales=F) == ALIGN
    assert norm(c, codes=F, scales=F + 4) == ALIGN
    none = dict.fromkeys(names)
    assert norm(c, T=0, **none) == M.MEP_OK         # no launch


def test_norm_backward_refusals():
    c = norm_cfg()
    token = norm_cfg(gate=M.MEP_BLOCK_GATE_TOKEN)
    assert backward(None) == NULL
    assert backward(c, T=-1) == SHAPE
    assert backward(c, ws=None) == NULL
    assert backward(c, gx=None, gy=None, gwp=None, gwn=None) == NULL  # nothing wanted
    assert backward(c, gs=None, gn=None, gwn=None) == NULL            # nothing to go by
    assert backward(c, s=None) == NULL
    assert backward(c, gn=None) == NULL                               # grad_pre_weight needs it
    assert backward(c, y=None) == NULL
    assert backward(token) == NULL
    assert backward(c, gate=F) == backward(c, gg=F) == CONFIG
    for name in ("gs", "gn", "s", "y", "wp", "bp", "wn", "gx", "gy", "gwp", "gbp", "gwn", "gbn", "ws"):
        assert backward(c, **{name: F + 8}) == ALIGN, name
    assert backward(token, gate=F + 4) == backward(token, gate=F, gg=F + 8) == ALIGN
    n = M.mep_block_norm_workspace_bytes(c, 4)
    assert n >= 4 * 7168 and backward(c, size=n - 1) == SHAPE
    assert M.mep_block_norm_workspace_bytes(c, -1) == 0
    assert M.mep_block_norm_workspace_bytes(c, 0) > 0
    assert M.mep_block_norm_workspace_bytes(c, 4096) >= n


def test_grad_refusals():
    ok = (F, F, 100, M.MEP_FP32)
    lib = M.lib()

    def both(rows, n=None, norm=F, ws=F, size=1 << 40, limit=1.0):
        a, m = grads(*rows)
        m = m if n is None else n
        return (lib.mep_grad_norm(a, m, norm, ws, size, None), lib.mep_grad_clip(a, m, norm, limit, None))

    assert both([ok], n=-1) == both([ok], n=65537) == (SHAPE, SHAPE)
    assert lib.mep_grad_norm(None, 1, F, F, 1 << 40, None) == NULL
    assert lib.mep_grad_clip(None, 1, F, 1.0, None) == NULL
    assert both([ok, (F, F, 8, 2)]) == (CONFIG, CONFIG)
    assert both([ok, (F, F, -1, 0)]) == both([ok, (F, F, (1 << 44) + 1, 0)]) == (SHAPE, SHAPE)
    assert both([ok], norm=None) == both([ok, (None, F, 8, 0)]) == (NULL, NULL)
    assert both([(F, F, 8, 0)], norm=F + 4) == both([(F + 8, F, 8, 0)]) == (ALIGN, ALIGN)
    assert lib.mep_grad_norm(*grads(ok), F, None, 1 << 40, None) == NULL
    assert lib.mep_grad_norm(*grads(ok), F, F + 8, 1 << 40, None) == ALIGN
    assert lib.mep_grad_norm(*grads(ok), F, F, 0, None) == SHAPE
    a, n = grads((F, None, 8, 0))
    assert lib.mep_grad_clip(a, n, F, 1.0, None) == NULL
    a, n = grads((F, F + 8, 8, 0))
    assert lib.mep_grad_clip(a, n, F, 1.0, None) == ALIGN
    a, n = grads(ok)
    a[0].reserved = 1
    assert lib.mep_grad_norm(a, n, F, F, 1 << 40, None) == lib.mep_grad_clip(a, n, F, 1.0, None) == CONFIG
    for limit in (0.0, -1.0, float("nan")):
        assert lib.mep_grad_clip(*grads(ok), F, limit, None) == CONFIG
    assert lib.mep_grad_clip(*grads((None, None, 0, 0)), F, 1.0, None) == M.MEP_OK  # nothing to do
    assert lib.mep_grad_clip(*grads(), F, 1.0, None) == M.MEP_OK


def test_grad_workspaces():
    lib = M.lib()
    assert lib.mep_grad_workspace_bytes(None, 1) == lib.mep_grad_workspace_bytes(None, -1) == 0
    one = lib.mep_grad_workspace_bytes(*grads((F, F, 100, 0)))
    many = lib.mep_grad_workspace_bytes(*grads(*[(F, F, 10 ** 6, 1)] * 500))
    assert 0 < lib.mep_grad_workspace_bytes(None, 0) <= one <= many
    assert lib.mep_grad_workspace_bytes(*grads((F, F, 100, 5))) == 0
    assert lib.mep_grad_workspace_bytes(*grads((F, F, 1 << 44, 0))) > 0


def test_binding_refuses_tensors():
    c = norm_cfg(hidden_dim=128)
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be torch.bfloat16"):
        M.mep_block_norm(c, x.float(), None, None, None, None, None, None, 4, None, x, None, None)
    with pytest.raises(ValueError, match="x holds"):
        M.mep_block_norm(c, x[:3], None, None, None, None, None, None, 4, None, x, None, None)
    with pytest.raises(ValueError, match="on the GPU"):
        M.mep_block_norm(c, x, None, None, None, None, None, None, 4, None, x, None, None)
    with pytest.raises(ValueError, match="n_codes must be"):
        M.mep_block_norm(c, F, None, None, None, None, None, None, 4, None, None, x.float(), F)
    with pytest.raises(ValueError, match="pre_weight must be torch.float32"):
        M.mep_block_norm_backward(c, F, F, F, None, None, None, None, x, 4, F, *[None] * 6, None)
    with pytest.raises(ValueError, match="logits holds"):
        M.mep_gate_grouped(gate_cfg(), 8, 4, M.MEP_GROUP_TOP2, torch.zeros((4, 255)), None, 4, F, F)
    with pytest.raises(ValueError, match="on the GPU"):
        M.MepGrads([torch.zeros(4)])
    with pytest.raises(ValueError, match="fp32 or bf16"):
        M.MepGrads([torch.zeros(4, dtype=torch.float16)])
    with pytest.raises(M.MepError) as e:
        M.mep_gate_grouped(gate_cfg(), 7, 4, M.MEP_GROUP_TOP2, F, None, 4, F, F, stream=0)
    assert e.value.code == CONFIG
    assert M.mep_grad_workspace_bytes(M.MepGrads([])) > 0
