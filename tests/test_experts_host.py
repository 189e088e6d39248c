"""Host-side checks of the router and expert calls (no GPU, nothing launched):
configs, sizes, null pointers, alignment, workspaces, and the binding's own
checks of tensors.  Device pointers are fake aligned addresses."""

import ctypes as C

import pytest
import torch

import combine_mep_plan_amd as M

F = 0x7F0000000000  # never dereferenced on the host


def gate_cfg(**kw):
    base = dict(num_experts=256, top_k=8, score=M.MEP_SCORE_SOFTMAX, dtype=M.MEP_FP32, normalize=1,
                scale=1.0, balance_coef=0.01)
    base.update(kw)
    return M.MepGateConfig(**base)


def lin_cfg(**kw):
    base = dict(num_experts=32, in_dim=7168, out_dim=2048, act=M.MEP_ACT_SILU_GLU,
                quant=M.MEP_QUANT_NONE)
    base.update(kw)
    return M.MepLinearConfig(**base)


def gate(c, logits=F, bias=None, T=4, indices=F, weights=F):
    return M.lib().mep_gate(C.byref(c) if c else None, logits, bias, T, indices, weights, None)


def balance(c, logits=F, indices=F, mask=None, T=4, counts=F, mean=F, loss=F, ws=F, n=1 << 40):
    return M.lib().mep_balance_loss(C.byref(c) if c else None, logits, indices, mask, T, counts,
                                    mean, loss, ws, n, None)


def gate_backward(c, logits=F, indices=F, mask=None, T=4, gw=F, counts=F, gl=F, out=F):
    return M.lib().mep_gate_backward(C.byref(c) if c else None, logits, indices, mask, T, gw,
                                     counts, gl, out, None)


def linear(c, x=F, xs=None, counts=F, off=F, cap=256, rows=8, w=F, ws=None, bias=None, res=None,
           y=F, z=None):
    return M.lib().mep_expert_linear(C.byref(c) if c else None, x, xs, counts, off, cap, rows, w,
                                     ws, bias, res, y, z, None)


def backward(c, gy=F, z=F, x=F, w=F, counts=F, off=F, cap=256, rows=8, gx=F, gw=F, gb=F, ws=F,
             n=1 << 40):
    return M.lib().mep_expert_linear_backward(C.byref(c) if c else None, gy, z, x, w, counts, off,
                                              cap, rows, gx, gw, gb, ws, n, None)


@pytest.mark.parametrize("bad", [dict(num_experts=0), dict(num_experts=4097), dict(top_k=0),
                                 dict(top_k=33), dict(num_experts=4, top_k=5), dict(score=2),
                                 dict(score=-1), dict(dtype=2)])
def test_bad_gate_configs(bad):
    c = gate_cfg(**bad)
    assert gate(c) == balance(c) == gate_backward(c) == M.MEP_ERR_CONFIG
    assert M.mep_balance_workspace_bytes(c, 4) == 0


@pytest.mark.parametrize("bad", [dict(num_experts=0), dict(num_experts=4097), dict(in_dim=0),
                                 dict(in_dim=12), dict(out_dim=-8), dict(out_dim=(1 << 20) + 8),
                                 dict(act=4), dict(act=-1), dict(quant=M.MEP_QUANT_MXFP4),
                                 dict(quant=M.MEP_QUANT_FP8_E4M3_BLOCK128, in_dim=72),
                                 dict(quant=M.MEP_QUANT_FP8_E4M3_BLOCK128, out_dim=200)])
def test_bad_linear_configs(bad):
    c = lin_cfg(**bad)
    assert linear(c, xs=F, ws=F) == backward(c) == M.MEP_ERR_CONFIG
    assert M.mep_linear_workspace_bytes(c, 256) == 0


def test_gate_refusals():
    c = gate_cfg()
    assert gate(None) == M.MEP_ERR_NULL
    assert gate(c, T=-1) == gate(c, T=(1 << 26) + 1) == M.MEP_ERR_SHAPE
    for kw in (dict(logits=None), dict(indices=None), dict(weights=None)):
        assert gate(c, **kw) == M.MEP_ERR_NULL
    for kw in (dict(logits=F + 4), dict(indices=F + 8), dict(weights=F + 4)):
        assert gate(c, **kw) == M.MEP_ERR_ALIGN
    assert gate(c, bias=F) == M.MEP_ERR_CONFIG      # a bias needs sigmoid scores
    assert gate(gate_cfg(score=M.MEP_SCORE_SIGMOID), bias=F + 4) == M.MEP_ERR_ALIGN
    assert gate(c, logits=None, indices=None, weights=None, T=0) == M.MEP_OK  # no launch


def test_balance_refusals():
    c = gate_cfg()
    n = M.mep_balance_workspace_bytes(c, 4)
    assert n > 0
    assert M.mep_balance_workspace_bytes(c, -1) == 0
    assert M.mep_balance_workspace_bytes(c, 4096) >= n
    assert balance(None) == M.MEP_ERR_NULL
    assert balance(c, T=-1) == M.MEP_ERR_SHAPE
    assert balance(gate_cfg(top_k=32), T=1 << 26) == M.MEP_ERR_SHAPE  # counts past int32
    assert balance(c, n=n - 1) == M.MEP_ERR_SHAPE
    for name in ("logits", "indices", "counts", "mean", "loss", "ws"):
        assert balance(c, **{name: None}) == M.MEP_ERR_NULL
        assert balance(c, **{name: F + 4}) == M.MEP_ERR_ALIGN
    assert balance(c, mask=F + 1) == M.MEP_ERR_ALIGN


def test_gate_backward_refusals():
    c = gate_cfg()
    assert gate_backward(None) == M.MEP_ERR_NULL
    assert gate_backward(c, T=-1) == M.MEP_ERR_SHAPE
    for kw in (dict(gw=None, counts=None, gl=None), dict(counts=None), dict(gl=None),
               dict(logits=None), dict(indices=None), dict(out=None)):
        assert gate_backward(c, **kw) == M.MEP_ERR_NULL
    for name in ("logits", "indices", "mask", "gw", "counts", "gl", "out"):
        assert gate_backward(c, **{name: F + 4}) == M.MEP_ERR_ALIGN
    assert gate_backward(c, T=0, logits=None, indices=None, out=None) == M.MEP_OK


def test_linear_refusals():
    c = lin_cfg()
    assert linear(None) == M.MEP_ERR_NULL
    assert linear(c, cap=-1) == linear(c, cap=1 << 31) == linear(c, rows=-1) == M.MEP_ERR_SHAPE
    for name in ("x", "counts", "off", "w", "y"):
        assert linear(c, **{name: None}) == M.MEP_ERR_NULL
    for name in ("x", "counts", "off", "w", "bias", "res", "y", "z"):
        assert linear(c, **{name: F + 8}) == M.MEP_ERR_ALIGN
    assert linear(c, x=None, w=None, y=None, cap=0) == M.MEP_OK
    f8 = lin_cfg(quant=M.MEP_QUANT_FP8_E4M3_BLOCK128)
    assert linear(f8, ws=F) == linear(f8, xs=F) == M.MEP_ERR_NULL
    assert linear(f8, xs=F + 4, ws=F) == linear(f8, xs=F, ws=F + 4) == M.MEP_ERR_ALIGN


def test_linear_backward_refusals():
    c = lin_cfg()
    n = M.mep_linear_workspace_bytes(c, 256)
    assert n >= 256 * 4096 * 2                       # grad_z in bf16
    assert M.mep_linear_workspace_bytes(c, -1) == 0
    assert 0 < M.mep_linear_workspace_bytes(lin_cfg(act=M.MEP_ACT_NONE), 256) < n
    assert backward(None) == M.MEP_ERR_NULL
    assert backward(lin_cfg(quant=M.MEP_QUANT_FP8_E4M3_BLOCK128)) == M.MEP_ERR_CONFIG
    assert backward(c, cap=-1) == backward(c, rows=-1) == backward(c, n=n - 1) == M.MEP_ERR_SHAPE
    for name in ("gy", "z", "x", "w", "counts", "off", "ws"):
        assert backward(c, **{name: None}) == M.MEP_ERR_NULL
    assert backward(c, gx=None, gw=None, gb=None) == M.MEP_ERR_NULL
    for name in ("gy", "z", "x", "w", "counts", "off", "gx", "gw", "gb", "ws"):
        assert backward(c, **{name: F + 8}) == M.MEP_ERR_ALIGN


def test_binding_checks_tensors():
    c = gate_cfg()
    f32, i32 = torch.float32, torch.int32
    z = lambda n, t=f32: torch.zeros(n, dtype=t)  # noqa: E731
    with pytest.raises(ValueError, match="logits must be torch.float32"):
        M.mep_gate(c, z(1024, torch.bfloat16), None, 4, z(32, i32), z(32))
    with pytest.raises(ValueError, match="logits holds"):
        M.mep_gate(c, z(1023), None, 4, z(32, i32), z(32))
    with pytest.raises(ValueError, match="indices must be torch.int32"):
        M.mep_gate(c, z(1024), None, 4, z(32, torch.int64), z(32))
    with pytest.raises(ValueError, match="weights holds"):
        M.mep_gate(c, z(1024), None, 4, z(32, i32), z(31))
    with pytest.raises(ValueError, match="counts holds"):
        M.mep_balance_loss(c, z(1024), z(32, i32), None, 4, z(256, i32), z(256), z(1),
                           z(8, torch.uint8))
    with pytest.raises(ValueError, match="token_mask holds"):
        M.mep_gate_backward(c, z(1024), z(32, i32), z(3, torch.uint8), 4, z(32), None, None,
                            z(1024))
    with pytest.raises(ValueError, match="on the GPU"):
        M.mep_gate(c, z(1024), None, 4, z(32, i32), z(32), stream=0)
    lc = lin_cfg(num_experts=2, in_dim=128, out_dim=128, act=M.MEP_ACT_NONE)
    b = torch.bfloat16
    ok = dict(x=z((256, 128), b), counts=z(2, i32), off=z(3, i32), w=z((2, 128, 128), b),
              y=z((256, 128), b))

    def call(**kw):
        a = {**ok, **kw}
        M.mep_expert_linear(lc, a["x"], None, a["counts"], a["off"], 256, 8, a["w"], None,
                            a.get("bias"), a.get("res"), a["y"], a.get("z"), stream=0)

    for name, bad, word in (("x", z((255, 128), b), "em_x holds"),
                            ("x", z((256, 128)), "em_x must be torch.bfloat16"),
                            ("off", z(2, i32), "em_offsets holds"),
                            ("w", z((2, 127, 128), b), "w holds"),
                            ("bias", z((2, 128), b), "bias must be torch.float32"),
                            ("res", z((255, 128), b), "residual holds"),
                            ("z", z((255, 128), b), "z holds"),
                            ("y", z((256, 127), b), "y holds")):
        with pytest.raises(ValueError, match=word):
            call(**{name: bad})
    with pytest.raises(ValueError, match="on the GPU"):
        call()
    with pytest.raises(ValueError, match="grad_w holds"):
        M.mep_expert_linear_backward(lc, ok["y"], None, ok["x"], ok["w"], ok["counts"], ok["off"],
                                     256, 8, None, z((2, 127, 128), b), None, z(8, torch.uint8))
