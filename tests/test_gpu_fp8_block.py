"""Experts in e4m3 with one scale per block of 128, and the layer around them.

Tolerance of the grouped FFN: the reference gives, per output, the 64-bit value
and a bound on what fp32 sums and the codes of H that lie within such a sum's
error of a rounding border can change (block_reference.ffn); the gate's product
adds 2^-24 and the bf16 rounding 2^-8 of the value.
"""
import math

import pytest
import torch

from mixture_experts_layer_49_b200 import native as nat
from mixture_experts_layer_49_b200 import synthetic as syn

import block_reference as ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


def quantize(x, sld, dev):
    T, d = x.shape
    codes = torch.empty((T, d), dtype=torch.uint8, device=dev)
    scale = torch.zeros((T, sld // 4), device=dev)
    nat.moe_quantize_rows_block(x, codes, scale)
    return codes, scale


def test_quantize_rows(cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(1)
    for T, d in ((1, 8), (3, 120), (5, 128), (7, 1032), (300, 2048), (33, 272)):
        x = (torch.randn((T, d), generator=g, device=cuda_device) *
             torch.exp2(torch.randint(-40, 40, (T, 1), generator=g, device=cuda_device).float())).bfloat16()
        x[0, :min(d, 128)] = 0
        if T > 1:
            x[1] = 1e-38
        ld_in, ld_out, ld_s = d + 16, d + 8, ((d + 127) // 128 + 2) * 4
        wide = torch.full((T, ld_in), 99.0, dtype=torch.bfloat16, device=cuda_device)
        wide[:, :d] = x
        codes = torch.full((T, ld_out), 7, dtype=torch.uint8, device=cuda_device)
        scale = torch.full((T, ld_s // 4), -7.0, device=cuda_device)
        nat.moe_quantize_rows_block(wide, codes, scale, cols=d)
        nb = (d + 127) // 128
        assert (codes[:, d:] == 7).all() and (scale[:, nb:] == -7).all()
        top = ref.block_max(x.cpu().double())
        want_s = (top.float() / 448.0)
        assert torch.equal(scale[:, :nb].cpu(), want_s)                     # fp32, correctly rounded
        # a true quotient: 448.0 / tensor multiplies by a rounded reciprocal
        inv = ref.spread(torch.div(torch.full_like(top, 448.0, dtype=torch.float32), top.float()), d)
        assert torch.equal(codes[:, :d].cpu(), (x.cpu().float() * inv).to(torch.float8_e4m3fn).view(torch.uint8))


def grouped(cfg, rows, counts, w, sld, dev, seed, gelu, shared=None):
    """One call on random packed rows; returns what check() needs."""
    g = torch.Generator(device=dev).manual_seed(seed)
    total, d = cfg.T * cfg.top_k, cfg.d_model
    x = torch.randn((total, d), generator=g, device=dev).bfloat16()
    x8, xs = quantize(x, sld, dev)
    offsets = torch.zeros(cfg.E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.tensor(counts, device=dev).cumsum(0)
    gate = torch.rand(total, generator=g, device=dev) + 0.25
    y = torch.full((nat.perm_rows(cfg), d), 776.0, dtype=torch.bfloat16, device=dev)
    ws = nat.alloc_workspace(cfg)
    xt8 = xts = None
    if cfg.d_ff_shared:
        xt8, xts = quantize(torch.randn((cfg.T, d), generator=g, device=dev).bfloat16(), sld, dev)
    ex = nat.fp8_block_experts(w, sld)
    nat.moe_grouped_ffn_fp8_block(cfg, x8, xs, offsets, gate, ex, w.get("b1"), w.get("b2"), xt8, xts, y, ws)
    assert nat.moe_get_device_status(ws) == nat.MOE_OK
    return dict(x8=x8, xs=xs, gate=gate, y=y, xt8=xt8, xts=xts, offsets=offsets, ws=ws, ex=ex)


def check(cfg, counts, w, r, far=False):
    h = {k: v.cpu() for k, v in w.items()}
    y = r["y"].cpu().double()
    x = ref.dequantize(r["x8"].cpu(), r["xs"].cpu())
    gate = r["gate"].cpu().double().unsqueeze(1)
    at, total = 0, cfg.T * cfg.top_k
    names = ("W1", "Wu", "W2")
    for e, n in enumerate(counts):
        if n == 0:
            continue
        m = [ref.dequantize_weight(h[k][e], h[k + "_scale"][e]) if k in h else None for k in names]
        b = (h["b1"][e], h["b2"][e]) if "b1" in h else (None, None)
        want, err = ref.ffn(x[at:at + n], *m, *b, far)
        want, err = want * gate[at:at + n], err * gate[at:at + n]
        off = (y[at:at + n] - want).abs()
        assert (off <= want.abs() * HALF * (1 + 2.0 ** -15) + err * (1 + HALF) + 1e-30).all(), (e, (off - err).max())
        at += n
    assert (y[at:total] == 776.0).all()                                     # rows behind the last group
    if cfg.d_ff_shared:
        m = [ref.dequantize_weight(h[k], h[k + "_scale"]) if k in h else None for k in ("Wsg", "Wsu", "Wsd")]
        want, err = ref.ffn(ref.dequantize(r["xt8"].cpu(), r["xts"].cpu()), *m, None, None)
        assert ((y[total:] - want).abs() <= want.abs() * HALF * (1 + 2.0 ** -15) + err * (1 + HALF) + 1e-30).all()


CASES = [
    # T, d, E, F, k, act, S, counts
    (1, 128, 4, 128, 2, "swiglu", 0, [1, 0, 0, 1]),
    (1, 256, 2, 256, 1, "gelu", 0, [0, 1]),
    (5, 16, 3, 16, 2, "swiglu", 16, [3, 0, 7]),
    (130, 272, 5, 144, 2, "gelu", 0, [0, 130, 1, 128, 1]),
    (300, 1040, 3, 400, 1, "swiglu", 0, [129, 0, 171]),
    (129, 512, 4, 768, 2, "swiglu", 272, [0, 258, 0, 0]),
    (128, 384, 2, 640, 2, "gelu", 896, [256, 0]),
    (70, 2048, 8, 128, 4, "swiglu", 0, [35, 3, 0, 100, 60, 2, 80, 0]),
    (40, 144, 2, 2064, 1, "swiglu", 0, [17, 12]),                            # capacity dropped 11 rows
    (64, 256, 2, 256, 2, "swiglu", 0, [0, 0]),                               # no row kept
    (600, 256, 3, 272, 2, "swiglu", 128, [257, 384, 513]),
    # a few tokens: one pass of eight rows, more rows than tokens, widths that end inside a block
    (8, 2048, 64, 768, 8, "swiglu", 0, [1] * 64),
    (8, 272, 3, 144, 2, "gelu", 272, [9, 0, 7]),
    (3, 1040, 40, 400, 2, "swiglu", 16, [0] * 33 + [1, 0, 3, 0, 0, 0, 2]),
    (7, 400, 8, 272, 8, "swiglu", 0, [33, 20, 0, 0, 0, 0, 1, 0]),
    (9, 272, 3, 144, 2, "gelu", 272, [9, 0, 9]),
    # one and two tokens: single rows, all rows on one expert (more than one pass), none kept
    (1, 2048, 64, 768, 8, "swiglu", 0, [1] * 8 + [0] * 56),
    (2, 2048, 64, 768, 8, "swiglu", 0, [0] * 40 + [1, 2] * 5 + [0] * 14),
    (2, 272, 8, 144, 8, "gelu", 272, [9, 0, 0, 0, 0, 0, 0, 7]),
    (2, 400, 8, 272, 8, "swiglu", 16, [0, 16, 0, 0, 0, 0, 0, 0]),
    (2, 1040, 40, 2064, 2, "swiglu", 16, [0] * 33 + [1, 0, 2, 0, 0, 0, 0]),
    (2, 16, 2, 16, 1, "gelu", 0, [0, 0]),
]


@pytest.mark.parametrize("T,d,E,F,k,act,S,counts", CASES)
def test_grouped_ffn(cuda_device, T, d, E, F, k, act, S, counts):
    wl = syn.Workload("block", T=T, d_model=d, E=E, d_ff=F, top_k=k, act=act, d_ff_shared=S)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg) + (16 if d == 272 else 0)                   # a wider stride too
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device, seed=2)
    r = grouped(cfg, None, counts, w, sld, cuda_device, T + d, act == "gelu")
    check(cfg, counts, w, r)


# thousands of tiles in one of the products, with last blocks of 1, 127, 128, 129
# and more rows, experts without rows, the shared expert and biases
@pytest.mark.parametrize("T,d,E,F,k,act,S,counts", [
    (4600, 144, 5, 2064, 2, "swiglu", 272, [4000, 129, 0, 4815, 256]),
    (15000, 1040, 5, 144, 2, "swiglu", 144, [29000, 1, 127, 700, 0]),
    (17400, 144, 4, 2064, 1, "gelu", 0, [17000, 130, 14, 256]),
    (31000, 1040, 4, 144, 1, "gelu", 0, [29900, 0, 900, 128]),
])
def test_grouped_ffn_of_many_rows(cuda_device, T, d, E, F, k, act, S, counts):
    test_grouped_ffn(cuda_device, T, d, E, F, k, act, S, counts)


def test_scales_of_every_block_count(cuda_device):
    """Scales spread over 2^-20 .. 2^20: a block scaled by a neighbour's scale would
    be far off."""
    wl = syn.Workload("block", T=140, d_model=400, E=2, d_ff=272, top_k=1)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device, seed=3)
    g = torch.Generator(device=cuda_device).manual_seed(9)
    for name in ("W1_scale", "Wu_scale", "W2_scale"):
        w[name] *= torch.exp2(torch.randint(-10, 11, w[name].shape, generator=g, device=cuda_device).float())
    check(cfg, [139, 1], w, grouped(cfg, None, [139, 1], w, sld, cuda_device, 5, False))


def test_bad_offsets_are_recorded(cuda_device):
    wl = syn.Workload("block", T=64, d_model=256, E=3, d_ff=256, top_k=1)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device)
    r = grouped(cfg, None, [20, 20, 24], w, sld, cuda_device, 1, False)
    good = r["y"].clone()
    for bad in ([0, 20, 10, 64], [-5, 20, 40, 64], [0, 20, 40, 65]):
        r["offsets"].copy_(torch.tensor(bad, dtype=torch.int32))
        r["y"].fill_(776.0)
        nat.moe_grouped_ffn_fp8_block(cfg, r["x8"], r["xs"], r["offsets"], r["gate"], r["ex"], None, None, None, None,
                                      r["y"], r["ws"])
        assert nat.moe_get_device_status(r["ws"]) == nat.MOE_ERR_DEVICE_BOUNDS
    r["offsets"].copy_(torch.tensor([0, 20, 40, 64], dtype=torch.int32))
    nat.moe_grouped_ffn_fp8_block(cfg, r["x8"], r["xs"], r["offsets"], r["gate"], r["ex"], None, None, None, None,
                                  r["y"], r["ws"])
    assert nat.moe_get_device_status(r["ws"]) == nat.MOE_OK and torch.equal(r["y"], good)


def test_infinite_and_nan_rows_stay_alone(cuda_device):
    wl = syn.Workload("block", T=200, d_model=256, E=2, d_ff=256, top_k=1)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device)
    r = grouped(cfg, None, [150, 50], w, sld, cuda_device, 1, False)
    want = r["y"].clone()
    r["x8"][7, 3] = 0x7F                                                     # a NaN code
    r["xs"][151, 0] = float("inf")
    nat.moe_grouped_ffn_fp8_block(cfg, r["x8"], r["xs"], r["offsets"], r["gate"], r["ex"], None, None, None, None,
                                  r["y"], r["ws"])
    keep = torch.ones(200, dtype=torch.bool)
    keep[[7, 151]] = False
    assert torch.equal(r["y"][keep.to(cuda_device)], want[keep.to(cuda_device)])
    assert torch.isnan(r["y"][7]).all() and not torch.isfinite(r["y"][151]).any()


def layer(cuda_device, T=300, groups=None, score="sigmoid", S=128, **kw):
    wl = syn.Workload("block_layer", T=T, d_model=272, E=16, d_ff=144, top_k=4, score=score, d_ff_shared=S,
                      sel_bias_std=0.1, **kw)
    cfg = nat.config_from_workload(wl)
    inp = syn.generate(wl, cuda_device, seed=1)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device, seed=1)
    return wl, cfg, inp, sld, w


@pytest.mark.parametrize("groups", [None, (4, 2, 2, 2.5)])
@pytest.mark.parametrize("cap", [0.0, 0.6])
def test_layer_equals_its_stages(cuda_device, groups, cap):
    """The whole layer, bit for bit, from its own stages: router, quantization,
    permute, grouped FFN, combine, statistics."""
    wl, cfg, inp, sld, w = layer(cuda_device, capacity_factor=cap)
    T, d, E, k = cfg.T, cfg.d_model, cfg.E, cfg.top_k
    grp = nat.route_groups(*groups) if groups else None
    out, ws = nat.Outputs(cfg), nat.alloc_workspace(cfg)
    nat.forward_fp8_block(cfg, inp, w, sld, out, ws, groups=grp)
    assert nat.moe_get_device_status(ws) == nat.MOE_OK
    i32 = dict(dtype=torch.int32, device=cuda_device)
    idx, gate = torch.empty((T, k), **i32), torch.empty((T, k), device=cuda_device)
    psum = torch.empty((nat.router_blocks(cfg), E), device=cuda_device)
    ws2 = nat.alloc_workspace(cfg)
    if grp:
        nat.moe_router_topk_groups(cfg, grp, inp["x"], inp["Wr"], None, inp["sel_bias"], idx, gate, None, psum, ws2)
    else:
        nat.moe_router_topk(cfg, inp["x"], inp["Wr"], None, inp["sel_bias"], idx, gate, None, psum, ws2)
    assert torch.equal(idx, out.idx) and torch.equal(gate, out.gate)
    counts, kept, offsets = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
    row_of, row_token = torch.empty((T, k), **i32), torch.empty(T * k, **i32)
    row_gate, x_perm = torch.zeros(T * k, device=cuda_device), torch.zeros((T * k, d), dtype=torch.bfloat16, device=cuda_device)
    dropped = torch.zeros(1, **i32)
    nat.moe_permute(cfg, inp["x"], idx, gate, counts, kept, offsets, row_of, row_token, row_gate, x_perm, dropped, ws2)
    x8p, xsp = quantize(x_perm, sld, cuda_device)
    x8, xs = quantize(inp["x"], sld, cuda_device)
    y_perm = torch.zeros((nat.perm_rows(cfg), d), dtype=torch.bfloat16, device=cuda_device)
    nat.moe_grouped_ffn_fp8_block(cfg, x8p, xsp, offsets, row_gate, nat.fp8_block_experts(w, sld), None, None, x8, xs,
                                  y_perm, ws2)
    y = torch.empty((T, d), dtype=torch.bfloat16, device=cuda_device)
    nat.moe_combine(cfg, y_perm, row_of, y, ws2)
    assert torch.equal(y, out.y) and torch.equal(counts, out.counts) and torch.equal(dropped, out.n_dropped)
    assert cap == 0.0 or dropped.item() > 0
    f, P, loss = torch.empty(E, device=cuda_device), torch.empty(E, device=cuda_device), torch.empty(1, dtype=torch.float64, device=cuda_device)
    nat.moe_balance_stats(cfg, counts, psum, f, P, loss)
    assert torch.equal(f, out.f) and torch.equal(P, out.P) and torch.equal(loss, out.loss)


def test_block_of_norm_routing_and_experts(cuda_device):
    """What a block runs: norm of the residual sum, its codes straight into the layer.
    The layer's output follows from the norm's own outputs in 64 bits."""
    wl, cfg, inp, sld, w = layer(cuda_device)
    T, d, k = cfg.T, cfg.d_model, cfg.top_k
    g = torch.Generator(device=cuda_device).manual_seed(4)
    res = (3.0 * torch.randn((T, d), generator=g, device=cuda_device)).bfloat16()
    branch = torch.randn((T, d), generator=g, device=cuda_device).bfloat16()
    wn = 1.0 + 0.1 * torch.randn(d, generator=g, device=cuda_device)
    groups = nat.route_groups(4, 2, 2, 2.5)
    h, y = torch.empty_like(res), torch.empty_like(res)
    codes = torch.empty((T, d), dtype=torch.float8_e4m3fn, device=cuda_device)
    scale = torch.zeros((T, sld // 4), device=cuda_device)
    out, ws = nat.Outputs(cfg, want_logits=True), nat.alloc_workspace(cfg)
    ex = nat.fp8_block_experts(w, sld)

    def block():
        nat.moe_rmsnorm(branch, res, wn, 1e-6, h, y, codes, scale)
        nat.forward_fp8_block(cfg, dict(inp, x=y), ex, sld, out, ws, groups=groups, x8=codes, xs=scale)

    block()
    torch.cuda.synchronize()
    assert nat.moe_get_device_status(ws) == nat.MOE_OK
    idx = ref.select(out.logits.cpu(), inp["sel_bias"].cpu(), k, 4, 2, 2, "sigmoid")
    assert torch.equal(out.idx.cpu(), idx)
    gate = ref.gates(out.logits.cpu(), idx, "sigmoid", 1, 2.5)
    hw = {n: t.cpu() for n, t in w.items()}
    x = ref.dequantize(codes.view(torch.uint8).cpu(), scale.cpu())
    m = [ref.dequantize_weight(hw[n], hw[n + "_scale"]) for n in ("Wsg", "Wsu", "Wsd")]
    want, err = ref.ffn(x, *m, None, None)
    err = err + want.abs() * HALF                                            # rows of y_perm are bf16
    for e in range(cfg.E):
        t, s = (idx == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        m = [ref.dequantize_weight(hw[n][e], hw[n + "_scale"][e]) for n in ("W1", "Wu", "W2")]
        ye, ee = ref.ffn(x[t], *m, None, None)
        gt = gate[t, s].unsqueeze(1)
        want.index_add_(0, t, ye * gt)
        err.index_add_(0, t, ee * gt * (1 + HALF) + (ye * gt).abs() * (HALF + 2.0 ** -16))
    got = out.y.cpu().double()
    assert ((got - want).abs() <= want.abs() * HALF + err * (1 + 2.0 ** -7)).all()
    # replayed from a graph: the same bits
    first = [t.clone() for t in (h, y, out.y, out.idx, out.gate, out.loss)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    out.y.zero_(), h.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (h, y, out.y, out.idx, out.gate, out.loss)))


def test_layer_without_tokens_and_with_one(cuda_device):
    for T in (0, 1):
        wl, cfg, inp, sld, w = layer(cuda_device, T=T)
        out, ws = nat.Outputs(cfg), nat.alloc_workspace(cfg)
        for grp in (None, nat.route_groups(4, 2)):
            nat.forward_fp8_block(cfg, inp, w, sld, out, ws, groups=grp)
            assert nat.moe_get_device_status(ws) == nat.MOE_OK
            assert out.counts.sum().item() == T * cfg.top_k and out.n_dropped.item() == 0


def test_group_limited_training(cuda_device):
    """Forward, training forward and backward with groups: the bf16 layer on the same
    choice of experts.  Without a factor the gradients equal those of the plain
    backward fed this choice; with a factor c on the gates the expert gradients
    and the task part of dx scale by c (here 2, exactly)."""
    wl = syn.Workload("group_train", T=96, d_model=128, E=16, d_ff=64, top_k=4, score="sigmoid", sel_bias_std=0.1)
    cfg = nat.config_from_workload(wl)
    inp = syn.generate(wl, cuda_device, seed=3)
    dy = torch.randn((96, 128), device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(1)).bfloat16()
    ws, bws = nat.alloc_workspace(cfg), nat.alloc_backward_workspace(cfg)
    res = {}
    for c in (1.0, 2.0):
        grp = nat.route_groups(4, 2, 2, c)
        out, out2 = nat.Outputs(cfg, want_logits=True), nat.Outputs(cfg, want_logits=True)
        nat.forward(cfg, inp, out, ws, groups=grp)
        nat.forward_train(cfg, inp, out2, ws, bws, groups=grp)
        for a in ("y", "idx", "gate", "counts", "loss"):
            assert torch.equal(getattr(out, a), getattr(out2, a))
        assert torch.equal(out.idx.cpu(), ref.select(out.logits.cpu(), inp["sel_bias"].cpu(), 4, 4, 2, 2, "sigmoid"))
        grads = nat.backward(cfg, inp, out2, ws, dy, alpha=0.0, ws=bws, groups=grp)
        if c == 1.0:
            nat.forward_train(cfg, inp, out2, ws, bws, groups=grp)
            plain = nat.backward(cfg, inp, out2, ws, dy, alpha=0.0, ws=bws)
            for n in ("dx", "dWr", "dW1", "dWu", "dW2", "dlogit_bias"):
                assert torch.equal(grads[n], plain[n]), n
        res[c] = {n: t.clone() for n, t in grads.items() if t is not None}
    for n in ("dW1", "dWu", "dW2", "dx", "dWr"):
        a, b = res[1.0][n].double(), res[2.0][n].double()
        assert (b - 2 * a).norm() <= 2.0 ** -16 * b.norm() + 1e-30, n


# T, d, E, F, k, S: few tiles and many, in either product, with and without the shared
# expert, and the form for one and two tokens
@pytest.mark.parametrize("T,d,E,F,k,act,S", [
    (2000, 1040, 16, 400, 2, "swiglu", 0), (9000, 144, 8, 2064, 2, "swiglu", 272), (15000, 1040, 5, 272, 2, "swiglu", 144),
    (2000, 1040, 16, 400, 1, "gelu", 0), (2, 2048, 64, 768, 8, "swiglu", 768),
])
def test_repeated_calls_give_the_same_bits(cuda_device, T, d, E, F, k, act, S):
    """The two warps that share a hidden row's block exchange its maximum: a maximum
    read too early would change codes from call to call."""
    wl = syn.Workload("block", T=T, d_model=d, E=E, d_ff=F, top_k=k, act=act, d_ff_shared=S)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device, seed=6)
    counts = torch.bincount(torch.randint(0, E, (T * k,), generator=torch.Generator().manual_seed(T)), minlength=E).tolist()
    r = grouped(cfg, None, counts, w, sld, cuda_device, T, act == "gelu")
    first = r["y"].clone()
    assert torch.isfinite(first).all()
    for _ in range(20):
        r["y"].fill_(776.0)
        nat.moe_grouped_ffn_fp8_block(cfg, r["x8"], r["xs"], r["offsets"], r["gate"], r["ex"], w.get("b1"), w.get("b2"),
                                      r["xt8"], r["xts"], r["y"], r["ws"])
        assert torch.equal(r["y"], first)
    assert nat.moe_get_device_status(r["ws"]) == nat.MOE_OK


def test_one_workspace_for_every_batch(cuda_device):
    """A batch that shrinks keeps its workspace: the same bits as in one of its own."""
    big = None
    for T in (40, 3, 2, 1):
        wl, cfg, inp, sld, w = layer(cuda_device, T=T)
        if big is None:
            big = nat.alloc_workspace(cfg)
        out, own, ws = nat.Outputs(cfg), nat.Outputs(cfg), nat.alloc_workspace(cfg)
        nat.forward_fp8_block(cfg, inp, w, sld, out, big)
        nat.forward_fp8_block(cfg, inp, w, sld, own, ws)
        assert nat.moe_get_device_status(big) == nat.MOE_OK
        assert torch.equal(out.y, own.y) and torch.equal(out.idx, own.idx)


@pytest.mark.parametrize("T,E,S", [(1, 64, 0), (2, 64, 0), (1, 200, 128), (2, 33, 128), (3, 64, 0)])
def test_bad_offsets_of_few_tokens_are_recorded(cuda_device, T, E, S):
    """Wherever the bad entry stands: before, at and after the experts with rows."""
    wl = syn.Workload("block", T=T, d_model=256, E=E, d_ff=256, top_k=1, d_ff_shared=S)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device)
    r = grouped(cfg, None, [T] + [0] * (E - 1), w, sld, cuda_device, 1, False)
    good, offsets = r["y"].clone(), r["offsets"].clone()

    def call():
        nat.moe_grouped_ffn_fp8_block(cfg, r["x8"], r["xs"], r["offsets"], r["gate"], r["ex"], None, None, r["xt8"],
                                      r["xts"], r["y"], r["ws"])
        return nat.moe_get_device_status(r["ws"])

    for at in (0, 1, 2, 31, 32, E // 2, E - 1, E):
        for bad in (-1, T + 4) + ((T - 1,) if at > 1 else ()):
            r["offsets"].copy_(offsets)
            r["offsets"][at] = bad
            assert call() == nat.MOE_ERR_DEVICE_BOUNDS, (at, bad)
    r["offsets"].copy_(offsets)
    assert call() == nat.MOE_OK and torch.equal(r["y"], good)


def test_gelu_in_its_tails(cuda_device):
    """Zero weights and b1 alone: every block of 128 hidden values is one GELU value,
    which the second product (the identity) returns as 448 * scale.  b2 takes the
    exact value away, so y is the error, in the units of the value: GELU 49 * 2^-24,
    scale, product, sum and b2 one each: below 2^-18.
    One, two and more tokens give the same bits."""
    d = 2048
    first = None
    for T, sign in ((1, -1), (2, -1), (3, -1), (300, -1), (3, 1), (1, 1)):
        wl = syn.Workload("block", T=T, d_model=d, E=8, d_ff=d, top_k=1, act="gelu")
        cfg = nat.config_from_workload(wl)
        sld = nat.fp8_block_sld(cfg)
        w = syn.generate_fp8_block_experts(wl, sld, cuda_device)
        w["W1"].zero_(), w["W2"].zero_()
        i = torch.arange(d, device=cuda_device)
        w["W2"][:, i, i] = 0x38                                             # 1.0
        w["W2_scale"].fill_(1.0)
        v = sign * torch.linspace(0.01, 9.0, 8 * d // 128).view(8, -1)
        a = v.repeat_interleave(128, 1)
        h = 0.5 * a.double() * torch.erfc(-a.double() / math.sqrt(2.0))
        w["b1"], w["b2"] = a.to(cuda_device).contiguous(), (-h).float().to(cuda_device).contiguous()
        counts = [0] * 8
        got = []
        for e in range(8):
            counts[e] = T
            r = grouped(cfg, None, counts, w, sld, cuda_device, 1, True)
            r["gate"].fill_(1.0)
            nat.moe_grouped_ffn_fp8_block(cfg, r["x8"], r["xs"], r["offsets"], r["gate"], r["ex"], w["b1"], w["b2"], None,
                                          None, r["y"], r["ws"])
            assert (r["y"] == r["y"][:1]).all()
            got.append(r["y"][0].cpu().double())
            counts[e] = 0
        got = torch.stack(got)
        assert (got.abs() <= h.abs() * 2.0 ** -18).all(), (got / h).abs().max()
        if sign < 0:
            first = got if first is None else first
            assert torch.equal(got, first)


def test_scales_forty_binary_orders_apart(cuda_device):
    """Weight scales spread over 2^-20 .. 2^20."""
    wl = syn.Workload("block", T=140, d_model=400, E=2, d_ff=272, top_k=1)
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device, seed=4)
    g = torch.Generator(device=cuda_device).manual_seed(10)
    for name in ("W1_scale", "Wu_scale", "W2_scale"):
        w[name] *= torch.exp2(torch.randint(-20, 21, w[name].shape, generator=g, device=cuda_device).float())
    check(cfg, [139, 1], w, grouped(cfg, None, [139, 1], w, sld, cuda_device, 5, False), far=True)
    wl = syn.Workload("block", T=2, d_model=400, E=2, d_ff=272, top_k=1)     # and the form for few tokens
    cfg = nat.config_from_workload(wl)
    check(cfg, [1, 1], w, grouped(cfg, None, [1, 1], w, sld, cuda_device, 6, False), far=True)


@pytest.mark.parametrize("T", [2, 200])
def test_gelu_rows_that_are_not_finite_stay_alone(cuda_device, T):
    wl = syn.Workload("block", T=T, d_model=256, E=2, d_ff=256, top_k=1, act="gelu")
    cfg = nat.config_from_workload(wl)
    sld = nat.fp8_block_sld(cfg)
    w = syn.generate_fp8_block_experts(wl, sld, cuda_device)
    r = grouped(cfg, None, [T - 1, 1], w, sld, cuda_device, 1, True)
    want = r["y"].clone()
    for bad in ("nan", "inf"):
        x8, xs = r["x8"].clone(), r["xs"].clone()
        if bad == "nan":
            x8[T - 2, 3] = 0x7F
        else:
            xs[T - 2, 0] = float("inf")
        nat.moe_grouped_ffn_fp8_block(cfg, x8, xs, r["offsets"], r["gate"], r["ex"], w["b1"], w["b2"], None, None, r["y"],
                                      r["ws"])
        keep = torch.arange(T, device=cuda_device) != T - 2
        assert torch.equal(r["y"][keep], want[keep])
        assert torch.isnan(r["y"][T - 2]).all() if bad == "nan" else not torch.isfinite(r["y"][T - 2]).any()
