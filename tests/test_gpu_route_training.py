"""The layer's router gradient with group-limited routing against 64 bits, through
dlogit_bias: the sum over tokens of d ell / d logits.

Tolerance.  A gate's gradient <dy, E_e(x)> comes from dy times the gate and hidden
rows in bf16: 2^-8 each, and fp32 sums (2^-11 covers them and the SiLU), relative
to the magnitudes sum |dy| |W2| |h|.  Through the gates' normalisation that error
enters like the gradient itself.  The scores' __expf is off by at most
(2 + 1.2 |l|) 2^-23, with |l| <= 32 here and a dozen further roundings less than
2^-13 of the magnitudes.
"""
import math

import pytest
import torch

from mixture_experts_layer_49_b200 import native as nat
from mixture_experts_layer_49_b200 import synthetic as syn

import block_reference as ref

pytestmark = pytest.mark.gpu
MODES = [("sigmoid", 1), ("softmax", 1), ("softmax", 0)]


def gate_gradients(inp, idx, dy):
    """<dy_t, E_e(x_t)> per slot and the magnitudes that meet, in 64 bits."""
    h = {n: inp[n].cpu().double() for n in ("x", "W1", "Wu", "W2")}
    dg, size = (torch.empty(idx.shape, dtype=torch.float64) for _ in range(2))
    for t in range(idx.shape[0]):
        for s, e in enumerate(idx[t].tolist()):
            g, u = h["W1"][e] @ h["x"][t], h["Wu"][e] @ h["x"][t]
            a = g / (1 + torch.exp(-g)) * u
            dg[t, s] = dy[t] @ (h["W2"][e] @ a)
            size[t, s] = dy[t].abs() @ (h["W2"][e].abs() @ a.abs())
    return dg, size


def spread_of(s, idx, dgate, counts, alpha, score, renorm, scale):
    """The magnitudes that meet in each logit's gradient."""
    T, E = s.shape
    chosen = s.gather(1, idx)
    total = chosen.sum(1, keepdim=True) if (score == "sigmoid" or renorm) else torch.ones((T, 1), dtype=torch.float64)
    own = torch.zeros_like(s).scatter_add_(1, idx, dgate.abs() * scale / total)
    mean = (own * s).sum(1, keepdim=True)
    bal = alpha * E / T * counts.double() / (T * idx.shape[1])
    z = s.sum(1, keepdim=True)
    if score == "sigmoid":
        hit = torch.zeros_like(s).scatter_(1, idx, 1.0)
        return s * (1 - s) * (own + hit * mean / total + (bal + (bal * s).sum(1, keepdim=True) / z) / z)
    return s * (own + 2 * mean + bal + (bal * s).sum(1, keepdim=True))


def layer(dev, T, score, renorm, seed):
    wl = syn.Workload("route_train", T=T, d_model=128, E=16, d_ff=64, top_k=4, score=score, renorm=renorm, sel_bias_std=0.1)
    cfg = nat.config_from_workload(wl)
    inp = syn.generate(wl, dev, seed=seed)
    dy = torch.randn((T, 128), device=dev, generator=torch.Generator(device=dev).manual_seed(seed)).bfloat16()
    return cfg, inp, dy, nat.alloc_workspace(cfg), nat.alloc_backward_workspace(cfg), nat.Outputs(cfg, want_logits=True)


def check(inp, out, dy, grads, alpha, score, renorm, scale, rows):
    """dlogit_bias from the tokens `rows` (the others contribute nothing)."""
    idx, logits = out.idx.cpu().long(), out.logits.cpu().clone()
    live = torch.zeros(idx.shape[0], 1, dtype=torch.float64)
    live[rows] = 1.0
    logits[(live == 0).flatten()] = 0.0                         # any number: these rows are left out
    counts = out.counts.cpu()
    dg, size = gate_gradients(inp, idx, dy.cpu().double())
    want = (ref.route_backward(logits, idx, dg, counts, alpha, score, renorm, scale) * live).sum(0)
    s = ref.scores(logits, score)
    off = spread_of(s, idx, size * (2.0 ** -7 + 2.0 ** -11), counts, 0.0, score, renorm, scale)
    off = off + spread_of(s, idx, dg, counts, alpha, score, renorm, scale) * 2.0 ** -13
    got = grads["dlogit_bias"].cpu().double()
    assert ((got - want).abs() <= (off * live).sum(0)).all(), ((got - want).abs() / (off * live).sum(0)).max()
    for n in ("dx", "dWr", "dW1", "dWu", "dW2"):
        assert torch.isfinite(grads[n]).all(), n


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("alpha,scale", [(0.0, 1.0), (0.0, 2.5), (0.5, 2.5)])
@pytest.mark.parametrize("T", [1, 6])
def test_router_gradient_with_groups(cuda_device, T, alpha, scale, score, renorm):
    cfg, inp, dy, ws, bws, out = layer(cuda_device, T, score, renorm, 3 + T)
    groups = nat.route_groups(4, 2, 2, scale)
    nat.forward_train(cfg, inp, out, ws, bws, groups=groups)
    grads = nat.backward(cfg, inp, out, ws, dy, alpha=alpha, ws=bws, groups=groups)
    check(inp, out, dy, grads, alpha, score, renorm, scale, list(range(T)))


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("alpha", [0.0, 0.5])
def test_a_row_without_scores_contributes_nothing(cuda_device, alpha, score, renorm):
    """A token whose logits are all -inf (gates of 0, as the forward pass defines)."""
    cfg, inp, dy, ws, bws, out = layer(cuda_device, 6, score, renorm, 5)
    groups = nat.route_groups(4, 2, 2, 2.5)
    nat.forward_train(cfg, inp, out, ws, bws, groups=groups)
    out.logits[2] = -math.inf
    out.gate[2] = 0.0
    grads = nat.backward(cfg, inp, out, ws, dy, alpha=alpha, ws=bws, groups=groups)
    check(inp, out, dy, grads, alpha, score, renorm, 2.5, [0, 1, 3, 4, 5])


@pytest.mark.parametrize("alpha", [0.0, 0.5])
@pytest.mark.parametrize("offset", [-100.0, -88.5])
def test_rows_of_tiny_sigmoids(cuda_device, offset, alpha):
    """Tokens 2 and 4 get logits near `offset` from the forward pass itself: below
    -88.72 no score is left, just above it the quotients stay finite."""
    cfg, inp, dy, ws, bws, out = layer(cuda_device, 6, "sigmoid", 1, 7)
    inp["x"][:, 0] = 1.0
    inp["x"][[2, 4]] = 0.0
    inp["Wr"][0] = -offset
    inp["logit_bias"] = torch.full((16,), offset, device=cuda_device) + 0.01 * torch.arange(16, device=cuda_device)
    groups = nat.route_groups(4, 2, 2, 16.0)
    nat.forward_train(cfg, inp, out, ws, bws, groups=groups)
    assert (out.logits[[2, 4]] < offset + 0.2).all() and ((out.gate[2] == 0).all() == (offset < -88.72))
    grads = nat.backward(cfg, inp, out, ws, dy, alpha=alpha, ws=bws, groups=groups)
    for n, g in grads.items():
        assert g is None or torch.isfinite(g).all(), n
    if offset < -88.72:
        check(inp, out, dy, grads, alpha, "sigmoid", 1, 16.0, [0, 1, 3, 5])
