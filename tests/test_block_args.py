"""Argument checks of the operators around the experts (RMS norm, group-limited
routing, experts in e4m3 with a scale per block of 128), without a GPU: none of
these calls reaches a launch.  And the reference gradients against differences.
"""
import ctypes

import pytest
import torch

from mixture_experts_layer_49_b200 import native as nat
from mixture_experts_layer_49_b200 import synthetic as syn

import block_reference as ref

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = (nat.MOE_OK, nat.MOE_ERR_INVALID_ARG, nat.MOE_ERR_UNSUPPORTED,
                                       nat.MOE_ERR_WORKSPACE)


def at(n=1, off=0):
    return P(4096 * n + off)


# ---------------------------------------------------------------- RMS norm
def norm(dtype=nat.MOE_BF16, rows=4, d=256, x=at(), residual=at(2), weight=at(3), eps=1e-6, h=at(4), y=at(5),
         codes=at(6), scale=at(7), ld=16):
    return nat.lib().moe_rmsnorm(dtype, rows, d, x, residual, weight, eps, h, y, codes, scale, ld, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), INVALID), (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=12), UNSUPPORTED),
    (dict(d=32776), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(weight=None), INVALID), (dict(h=None, y=None, codes=None, scale=None), INVALID),
    (dict(codes=None), INVALID), (dict(scale=None), INVALID), (dict(ld=4), INVALID), (dict(ld=18), INVALID),
    (dict(x=at(1, 8)), INVALID), (dict(residual=at(1, 2)), INVALID), (dict(weight=at(1, 4)), INVALID),
    (dict(h=at(1, 8)), INVALID), (dict(y=at(1, 8)), INVALID), (dict(codes=at(1, 4)), INVALID),
    (dict(scale=at(1, 2)), INVALID), (dict(rows=0), OK), (dict(rows=0, x=None), OK),
])
def test_norm_arguments(kw, code):
    assert norm(**kw) == code, nat.last_error_detail()


def norm_bwd(dtype=nat.MOE_F32, rows=4, d=256, h=at(), weight=at(2), eps=1e-6, dy=at(3), dres=at(4), dh=at(5),
             dweight=at(6), ws=at(8), ws_bytes=1 << 20):
    return nat.lib().moe_rmsnorm_backward(dtype, rows, d, h, weight, eps, dy, dres, dh, dweight, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), INVALID), (dict(rows=-2), INVALID), (dict(d=20), UNSUPPORTED), (dict(h=None), INVALID),
    (dict(weight=None), INVALID), (dict(dy=None), INVALID), (dict(dh=None), INVALID), (dict(dweight=None), INVALID),
    (dict(dy=at(1, 8)), INVALID), (dict(dres=at(1, 8)), INVALID), (dict(dweight=at(1, 2)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=at(8, 16)), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
])
def test_norm_backward_arguments(kw, code):
    assert norm_bwd(**kw) == code, nat.last_error_detail()


def test_norm_backward_workspace_size():
    size = nat.lib().moe_rmsnorm_backward_workspace_size
    assert size(-1, 256) == 0 and size(4, 12) == 0 and size(4, 0) == 0
    assert size(4, 256) >= 4 * 256 * 4 and size(10 ** 6, 256) == size(10 ** 7, 256)
    with pytest.raises(nat.MoEError):
        nat.rmsnorm_backward_workspace_size(4, 12)
    assert norm_bwd(rows=4, d=256, ws_bytes=size(4, 256) - 1) == WORKSPACE


# ---------------------------------------------------------------- routing
def cfg(**kw):
    base = dict(T=64, d_model=128, E=8, d_ff=256, top_k=2)
    base.update({k: kw.pop(k) for k in list(kw) if k in base})
    return nat.make_config(base["T"], base["d_model"], base["E"], base["d_ff"], base["top_k"], **kw)


def select(c, g, logits=at(), bias=None, idx=at(2), gate=at(3), psum=at(4)):
    return nat.lib().moe_route_select(ctypes.byref(c), g and ctypes.byref(g), logits, bias, idx, gate, psum, None)


BAD_GROUPS = [(3, 1, 1, 1.0), (0, 1, 1, 1.0), (4, 0, 1, 1.0), (4, 5, 1, 1.0), (4, 2, 0, 1.0), (4, 2, 3, 1.0),
              (8, 2, 2, 1.0), (4, 2, 2, 0.0), (4, 2, 2, -1.0), (4, 2, 2, float("nan")), (4, 2, 2, float("inf"))]


@pytest.mark.parametrize("groups", BAD_GROUPS)
def test_bad_groups_are_rejected_everywhere(groups):
    c, g = cfg(), nat.route_groups(*groups)
    L, cp, gp = nat.lib(), ctypes.byref(c), ctypes.byref(g)
    assert select(c, g) == INVALID
    assert L.moe_route_backward(cp, gp, at(), at(2), at(3), at(4), 0.1, at(5), None) == INVALID
    assert L.moe_router_topk_groups(cp, gp, *[at()] * 9, nat.workspace_size(c), None) == INVALID
    assert L.moe_forward_groups(cp, gp, *[at()] * 22, nat.workspace_size(c), None) == INVALID
    assert L.moe_forward_train_groups(cp, gp, *[at()] * 22, nat.workspace_size(c), at(), 1 << 30, None) == INVALID
    assert L.moe_backward_groups(cp, gp, *[at()] * 15, 0.0, *[at()] * 11, at(), 1 << 30, at(), 1 << 30, None) == INVALID
    w = block_weights()
    assert block_forward(c, g, w) == INVALID


def test_too_few_experts_in_the_kept_groups():
    assert select(cfg(top_k=5), nat.route_groups(4, 2, 2)) == INVALID
    assert "top_k" in nat.last_error_detail()


def test_route_arguments():
    c, g = cfg(), nat.route_groups(4, 2, 2, 2.5)
    assert select(c, None) == INVALID
    for name in ("logits", "idx", "gate"):
        assert select(c, g, **{name: None}) == INVALID
        assert select(c, g, **{name: at(1, 2)}) == INVALID
    assert select(cfg(T=0), g, logits=None, idx=None, gate=None) == OK
    L = nat.lib()

    def back(c, logits=at(), idx=at(2), dgate=at(3), counts=at(4), alpha=0.1, dlogits=at(5)):
        return L.moe_route_backward(ctypes.byref(c), ctypes.byref(g), logits, idx, dgate, counts, alpha, dlogits, None)

    for name in ("logits", "idx", "dgate", "dlogits", "counts"):
        assert back(c, **{name: None}) == INVALID
    assert back(c, alpha=float("nan")) == INVALID
    assert back(cfg(T=0)) == OK
    assert L.moe_router_topk_groups(ctypes.byref(c), ctypes.byref(g), *[at()] * 8, at(9, 16), 1 << 30, None) == WORKSPACE
    assert L.moe_router_topk_groups(ctypes.byref(c), None, *[at()] * 9, 1 << 30, None) == INVALID


# ---------------------------------------------------------------- block-scaled experts
def block_weights(sld=16, **kw):
    f = dict(W1=4096, W1_scale=4096, Wu=4096, Wu_scale=4096, W2=4096, W2_scale=4096, sld=sld)
    f.update(kw)
    return nat.MoeFp8BlockExperts(**f)


def block_forward(c, g, w, ws_bytes=None, **null):
    args = dict(x=at(), x8=at(2), xs=at(3), Wr=at(), lb=None, sb=None)
    rest = dict(b1=None, b2=None, y=at(), idx=at(), gate=at(), counts=at(), f=at(), P=at(), loss=at(), logits=None,
                nd=None)
    for k, v in null.items():
        (args if k in args else rest)[k] = v
    return nat.lib().moe_forward_fp8_block(ctypes.byref(c), g and ctypes.byref(g), *args.values(),
                                           w and ctypes.byref(w), *rest.values(), at(16),
                                           nat.workspace_size(c) if ws_bytes is None else ws_bytes, None)


def block_ffn(c, w, **null):
    a = dict(x8=at(), xs=at(), off=at(), rg=at())
    b = dict(b1=None, b2=None, xt=None, xts=None, y=at())
    for k, v in null.items():
        (a if k in a else b)[k] = v
    return nat.lib().moe_grouped_ffn_fp8_block(ctypes.byref(c), *a.values(), w and ctypes.byref(w), *b.values(), at(16),
                                               nat.workspace_size(c), None)


def test_block_expert_arguments():
    c = cfg()
    assert block_ffn(c, None) == INVALID and block_forward(c, None, None) == INVALID
    for sld in (0, 4, 12, 24, -16):
        assert block_ffn(c, block_weights(sld)) == INVALID, sld
        assert block_forward(c, None, block_weights(sld)) == INVALID
    assert block_ffn(cfg(d_ff=1040), block_weights(32)) == INVALID          # 9 blocks need 36 bytes
    for kw in (dict(dtype="f32"), dict(d_model=136), dict(d_ff=264), dict(d_ff_shared=24)):
        assert block_ffn(cfg(**kw), block_weights()) == UNSUPPORTED
        assert block_forward(cfg(**kw), None, block_weights()) == UNSUPPORTED
    for name in ("W1", "W1_scale", "Wu", "Wu_scale", "W2", "W2_scale"):
        assert block_ffn(c, block_weights(**{name: None})) == INVALID
        assert block_ffn(c, block_weights(**{name: 4096 + 8})) == INVALID
    assert block_ffn(cfg(act="gelu"), block_weights(Wu=None, Wu_scale=None), y=None) == INVALID
    for name in ("x8", "xs", "off", "rg", "y"):
        assert block_ffn(c, block_weights(), **{name: None}) == INVALID
    assert block_ffn(c, block_weights(), x8=at(1, 8)) == INVALID
    s = cfg(d_ff_shared=128)
    assert block_ffn(s, block_weights()) == INVALID                          # no shared weights
    shared = dict(Wsh_g=4096, Wsh_g_scale=4096, Wsh_u=4096, Wsh_u_scale=4096, Wsh_d=4096, Wsh_d_scale=4096)
    assert block_ffn(s, block_weights(**shared)) == INVALID                  # no x8 / xs
    assert block_ffn(cfg(T=0), block_weights()) == OK


def test_block_forward_arguments():
    c, w = cfg(), block_weights()
    for name in ("x", "Wr", "y", "idx", "gate", "counts", "f", "P", "loss"):
        assert block_forward(c, None, w, **{name: None}) == INVALID, name
    assert block_forward(c, None, w, x8=None) == INVALID and "both or neither" in nat.last_error_detail()
    assert block_forward(c, None, w, xs=None) == INVALID
    assert block_forward(c, None, w, xs=at(3, 8)) == INVALID
    assert block_forward(c, None, w, ws_bytes=nat.workspace_size(c) - 1) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(cols=-8), INVALID), (dict(cols=12), UNSUPPORTED), (dict(ld_in=120), INVALID),
    (dict(ld_in=132), INVALID), (dict(ld_out=120), INVALID), (dict(ld_scale=0), INVALID), (dict(ld_scale=6), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scale=None), INVALID), (dict(x=at(1, 8)), INVALID),
    (dict(codes=at(1, 4)), INVALID), (dict(rows=0), OK),
])
def test_quantize_block_arguments(kw, code):
    a = dict(x=at(), rows=4, cols=128, ld_in=128, codes=at(2), ld_out=128, scale=at(3), ld_scale=4)
    a.update(kw)
    assert nat.lib().moe_quantize_rows_block(*a.values(), None) == code, nat.last_error_detail()


def test_binding_refuses_host_tensors_and_sizes():
    t = torch.zeros(4, 16, dtype=torch.bfloat16)
    c, g = cfg(), nat.route_groups(4, 2)
    with pytest.raises(ValueError):
        nat.moe_rmsnorm(t, None, torch.zeros(16), 1e-6, None, t)
    with pytest.raises(ValueError):
        nat.moe_route_select(c, g, torch.zeros(64, 8), None, torch.zeros(64, 2, dtype=torch.int32), torch.zeros(64, 2))
    with pytest.raises(ValueError):
        nat.fp8_block_experts(dict(W1=torch.zeros(8, 16, 16, dtype=torch.uint8)), 16)


def test_binding_refuses_experts_smaller_than_the_layer(monkeypatch):
    """Host tensors stand in for device tensors: no call gets as far as a launch."""
    monkeypatch.setattr(nat, "_current_device", lambda: -1)
    wl = syn.Workload("block", T=4, d_model=272, E=4, d_ff=144, top_k=1, d_ff_shared=16)
    c, sld = nat.config_from_workload(wl), 16
    full = syn.generate_fp8_block_experts(wl, sld)

    def ffn(w):
        nat.moe_grouped_ffn_fp8_block(c, None, None, None, None, nat.fp8_block_experts(w, sld), None, None, None, None, None,
                                      torch.zeros(256, dtype=torch.uint8))

    def forward(w):
        nat.moe_forward_fp8_block(c, None, *[None] * 6, nat.fp8_block_experts(w, sld), *[None] * 11,
                                  torch.zeros(256, dtype=torch.uint8))

    for name in ("W1", "Wu", "W2"):
        less = {name: full[name][:3].contiguous(), name + "_scale": full[name + "_scale"][:3].contiguous()}
        for call in (ffn, forward):
            with pytest.raises(ValueError, match=name):
                call(dict(full, **less))
    for name in ("Wsg", "Wsu", "Wsd"):
        less = {name: full[name][:, :8].contiguous()}
        for call in (ffn, forward):
            with pytest.raises(ValueError, match=name):
                call(dict(full, **less))
    short = dict(full, W2=full["W2"].reshape(4, 144, 272))                  # one block of rows fewer than its shape
    short["W2_scale"] = full["W2_scale"][:, :2].contiguous()
    for call in (ffn, forward):
        with pytest.raises(ValueError, match="W2_scale"):
            call(short)


def test_scale_row_stride():
    assert nat.fp8_block_sld(cfg()) == 16
    assert nat.fp8_block_sld(cfg(d_model=7168)) == 224
    assert nat.fp8_block_sld(cfg(d_ff=1040)) == 48
    wl = syn.Workload("block", T=4, d_model=272, E=2, d_ff=144, top_k=1, d_ff_shared=16)
    w = syn.generate_fp8_block_experts(wl, 16)
    assert w["W1"].shape == (2, 144, 272) and w["W1_scale"].shape == (2, 2, 4) and w["W2_scale"].shape == (2, 3, 4)
    assert w["Wsd"].shape == (272, 16) and w["Wsd_scale"].shape == (3, 4)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("d,F,E,k,S", [(4096, 14336, 8, 2, 0), (2048, 8192, 8, 2, 0), (2048, 768, 128, 8, 0),
                                       (7168, 2048, 32, 8, 2048), (128, 2048, 4, 1, 4096), (128, 256, 8, 2, 0)])
def test_a_workspace_of_more_tokens_serves_fewer(d, F, E, k, S, act):
    """One workspace for the largest batch: the size never falls as tokens are added."""
    sizes = [nat.workspace_size(nat.make_config(T, d, E, F, k, act=act, d_ff_shared=S)) for T in range(300)]
    assert sizes == sorted(sizes) and sizes[0] > 0


# ---------------------------------------------------------------- reference gradients against differences
def test_norm_gradient_is_the_difference_quotient():
    g = torch.Generator().manual_seed(3)
    h, dy = (torch.randn((3, 24), generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(24, generator=g, dtype=torch.float64)
    dres = torch.randn((3, 24), generator=g, dtype=torch.float64)
    dh, dw, _, _ = ref.rmsnorm_backward(h, w, 1e-6, dy, dres)
    step = 2.0 ** -17                      # truncation and rounding both near 2^-34

    def loss(h, w):
        return (ref.rmsnorm(h, None, w, 1e-6)[1] * dy).sum() + (dres * h).sum()

    for i in range(h.numel()):
        e = torch.zeros(h.numel(), dtype=torch.float64)
        e[i] = step
        e = e.view_as(h)
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - dh.flatten()[i]) < 1e-8
    for i in range(24):
        e = torch.zeros(24, dtype=torch.float64)
        e[i] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[i]) < 1e-8


@pytest.mark.parametrize("score,renorm", [("softmax", 0), ("softmax", 1), ("sigmoid", 1)])
def test_route_gradient_is_the_difference_quotient(score, renorm):
    g = torch.Generator().manual_seed(5)
    l = torch.randn((4, 12), generator=g, dtype=torch.float64)
    idx = ref.select(l, None, 3, 4, 2, 2, score)
    dgate = torch.randn((4, 3), generator=g, dtype=torch.float64)
    counts = torch.bincount(idx.flatten().long(), minlength=12)
    args = (idx, dgate, counts, 0.3, score, renorm, 2.5)
    dl = ref.route_backward(l, *args)
    step = 2.0 ** -17
    for i in range(l.numel()):
        e = torch.zeros(l.numel(), dtype=torch.float64)
        e[i] = step
        e = e.view_as(l)
        diff = (ref.route_loss(l + e, *args) - ref.route_loss(l - e, *args)) / (2 * step)
        assert abs(diff - dl.flatten()[i]) < 1e-8
