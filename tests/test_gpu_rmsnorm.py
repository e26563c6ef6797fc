"""RMS norm with the residual's addition and an 8-bit output, forward and
backward, against 64 bits.

Tolerances.  fp32 arithmetic before a rounding: the sum of squares adds d terms
over threads of at most 32 values, 5 shuffles and at most 32 warps, so it is
off by at most 70 roundings of 2^-24, its root by half of that; mean, eps, root,
and three products add at most 8 more: 43 * 2^-24 < 2^-18 relative.  Then half a
step of the output's type: 2^-8 (bf16), 2^-24 (fp32), and for the codes 2^-4 of
the value or 2^-10 (half the smallest code) of a scale.
"""
import pytest
import torch

from mixture_experts_layer_49_b200 import native as nat

import block_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6
FP32 = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rows_of(T, d, dt, dev, seed, loud=True):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((T, d), generator=g, device=dev)
    if loud:
        x[:, ::97] *= 30.0
    return x.to(dt)


def call(x, r, w, eps=EPS, want=("h", "y", "q"), pad=0):
    T, d = x.shape
    nb = (d + 127) // 128
    h = torch.empty_like(x) if "h" in want else None
    y = torch.empty_like(x) if "y" in want else None
    codes = torch.empty((T, d), dtype=torch.uint8, device=x.device) if "q" in want else None
    scale = torch.full((T, nb + pad), -7.0, device=x.device) if "q" in want else None
    nat.moe_rmsnorm(x, r, w, eps, h, y, codes, scale)
    return h, y, codes, scale


def check(x, r, w, out, eps=EPS):
    h, y, codes, scale = out
    half = HALF[x.dtype]
    z, v = ref.rmsnorm(x.cpu(), None if r is None else r.cpu(), w.cpu(), eps)
    if h is not None:
        assert ((h.cpu().double() - z).abs() <= z.abs() * (half + 2.0 ** -24)).all()
    if y is not None:
        assert ((y.cpu().double() - v).abs() <= v.abs() * (half * (1 + FP32) + FP32) + 1e-38).all()
    if codes is not None:
        nb = (x.shape[1] + 127) // 128
        s = scale.cpu().double()
        want = ref.block_max(v) / 448.0
        assert ((s[:, :nb] - want).abs() <= want * (FP32 + 2.0 ** -22)).all()
        assert (s[:, nb:] == -7.0).all()                       # behind the last block: untouched
        sc = ref.spread(s[:, :nb], x.shape[1])
        got = codes.cpu().view(torch.float8_e4m3fn).double() * sc
        tol = torch.maximum(v.abs() * 2.0 ** -4, sc * 2.0 ** -10) + (v.abs() + sc * 448) * 2 * FP32
        assert ((got - v).abs() <= tol).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 2048), (3, 120), (5, 128), (7, 136), (33, 256), (130, 520), (9, 1032),
                                 (17, 2056), (4, 4104), (6, 7168), (3, 8200), (2, 16384), (2, 32768), (1000, 64)])
def test_norm(cuda_device, T, d, dt):
    x, r = rows_of(T, d, dt, cuda_device, 1, loud=False), rows_of(T, d, dt, cuda_device, 2)
    w = 1.0 + 0.1 * torch.randn(d, device=cuda_device)
    check(x, r, w, call(x, r, w, pad=3))
    check(x, None, w, call(x, None, w))


@pytest.mark.parametrize("want", [("h",), ("y",), ("q",), ("h", "q"), ("y", "q"), ("h", "y")])
def test_any_output_may_be_left_out(cuda_device, want):
    x, r = rows_of(70, 392, torch.bfloat16, cuda_device, 3), rows_of(70, 392, torch.bfloat16, cuda_device, 4)
    w = torch.rand(392, device=cuda_device) + 0.5
    full, part = call(x, r, w), call(x, r, w, want=want)
    check(x, r, w, part)
    for a, b in zip(full, part):
        assert b is None or torch.equal(a, b)


def test_in_place(cuda_device):
    for d in (256, 4104):
        x, r = rows_of(50, d, torch.bfloat16, cuda_device, 5), rows_of(50, d, torch.bfloat16, cuda_device, 6)
        w = torch.rand(d, device=cuda_device) + 0.5
        h, y, _, _ = call(x, r, w)
        x2, r2 = x.clone(), r.clone()
        nat.moe_rmsnorm(x2, r2, w, EPS, r2, x2)                # h into the residual, y into x
        assert torch.equal(r2, h) and torch.equal(x2, y)


def test_small_and_special_values(cuda_device):
    d = 384
    w = torch.ones(d, device=cuda_device)
    x = torch.zeros((6, d), device=cuda_device)
    x[1] = 1e-30                                               # mean square underflows beside eps
    x[2, 5] = 3.0                                              # two blocks of zeros
    x[3] = torch.linspace(-1e-20, 1e-20, d, device=cuda_device)
    x[4, 7] = float("nan")
    x[5, 9] = float("inf")
    _, y, codes, scale = call(x, None, w)
    check(x[:4], None, w, (None, y[:4], codes[:4], scale[:4]))
    assert (codes[0] == 0).all() and torch.isfinite(scale[:4]).all() and (scale[:4] > 0).all()
    assert torch.isnan(y[4]).all()
    assert torch.isnan(y[5, 9]) and (y[5, :9] == 0).all()
    # nothing of the special rows reaches the others
    assert torch.equal(call(x[:4].contiguous(), None, w)[1], y[:4])


def test_no_rows(cuda_device):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=cuda_device)
    w = torch.ones(256, device=cuda_device)
    call(x, None, w)
    dw = torch.full((256,), 5.0, device=cuda_device)
    nat.moe_rmsnorm_backward(x, w, EPS, x, None, torch.empty_like(x), dw,
                             nat.alloc_rmsnorm_backward_workspace(0, 256))
    assert (dw == 0).all()


def backward(h, w, dy, dres, eps=EPS, ws=None):
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    if ws is None:
        ws = nat.alloc_rmsnorm_backward_workspace(*h.shape)
    nat.moe_rmsnorm_backward(h, w, eps, dy, dres, dh, dw, ws)
    return dh, dw


# dh: two sums over the row (uh needs one more product per term) and at most
# twelve further roundings, each relative to the magnitudes that meet:
# 2^-17 of them.  dw: each block adds at most ceil(T / 592) rows in turn, the
# second pass at most 74 + 8 partial sums, n carries 2^-18.
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 2048), (3, 120), (5, 136), (33, 256), (700, 520), (1500, 64), (17, 2056),
                                 (600, 4104), (6, 7168), (3, 8200), (2, 16384), (2, 32768)])
def test_norm_backward(cuda_device, T, d, dt):
    h, dy, dres = (rows_of(T, d, dt, cuda_device, s, loud=s == 7) for s in (7, 8, 9))
    w = 1.0 + 0.1 * torch.randn(d, device=cuda_device)
    for res in (dres, None):
        dh, dw = backward(h, w, dy, res)
        want, wantw, size, sizew = ref.rmsnorm_backward(h.cpu(), w.cpu(), EPS, dy.cpu(),
                                                        None if res is None else res.cpu())
        assert ((dh.cpu().double() - want).abs() <= want.abs() * HALF[dt] * (1 + 2.0 ** -16) + size * 2.0 ** -17).all()
        adds = -(-T // 592) + 82
        assert ((dw.cpu().double() - wantw).abs() <= sizew * (adds * 2.0 ** -24 + FP32)).all()


def test_backward_is_deterministic_and_in_place(cuda_device):
    h, dy, dres = (rows_of(3000, 1032, torch.bfloat16, cuda_device, s) for s in (1, 2, 3))
    w = torch.rand(1032, device=cuda_device) + 0.5
    dh, dw = backward(h, w, dy, dres)
    ws = torch.full((nat.rmsnorm_backward_workspace_size(3000, 1032),), 255, dtype=torch.uint8, device=cuda_device)
    again = backward(h, w, dy, dres, ws=ws)                    # scratch full of NaN
    assert torch.equal(dh, again[0]) and torch.equal(dw, again[1])
    a, b = dy.clone(), dres.clone()
    nat.moe_rmsnorm_backward(h, w, EPS, a, dres, a, torch.empty_like(w), ws)
    nat.moe_rmsnorm_backward(h, w, EPS, dy, b, b, torch.empty_like(w), ws)
    assert torch.equal(a, dh) and torch.equal(b, dh)


def test_gradient_against_differences_of_the_kernel(cuda_device):
    """fp32 rows: the directional difference quotient of sum(y * dy) along unit-size
    directions.  Step 2^-6: truncation |f'''| 2^-12 / 6 with |f'''| of the order of
    the gradient's terms; y is off by 2^-18, so the sum of N terms by at most
    N 2^-18 max|y dy|, far more than random rounding gives; 2^-6 * 2 divides it."""
    T, d, step = 4, 256, 2.0 ** -6
    h, dy, p = (rows_of(T, d, torch.float32, cuda_device, s, loud=False) for s in (1, 2, 3))
    w = torch.rand(d, device=cuda_device) + 0.5
    dh, _ = backward(h, w, dy, None)
    f = lambda x: (call(x, None, w, want=("y",))[1].double() * dy.double()).sum().item()
    got = (f(h + step * p) - f(h - step * p)) / (2 * step)
    want = (dh.double() * p.double()).sum().item()
    size = (dh.double() * p.double()).abs().sum().item()
    terms = (call(h, None, w, want=("y",))[1].double() * dy.double()).abs().sum().item()
    assert abs(got - want) <= terms * 2.0 ** -18 / step + size * 2.0 ** -12 * 8


def test_graph_streams_and_refusals(cuda_device):
    x, r = rows_of(40, 512, torch.bfloat16, cuda_device, 5), rows_of(40, 512, torch.bfloat16, cuda_device, 6)
    w = torch.rand(512, device=cuda_device) + 0.5
    want = call(x, r, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, y = torch.empty_like(x), torch.empty_like(x)
    nat.moe_rmsnorm(x, r, w, EPS, h, y, stream=side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    dh, dw, ws = torch.empty_like(x), torch.empty_like(w), nat.alloc_rmsnorm_backward_workspace(40, 512)
    h.zero_(), y.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nat.moe_rmsnorm(x, r, w, EPS, h, y)
        nat.moe_rmsnorm_backward(h, w, EPS, y, r, dh, dw, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    ref_dh, ref_dw = backward(want[0], w, want[1], r)
    assert torch.equal(dh, ref_dh) and torch.equal(dw, ref_dw)
    for bad in (dict(x=x.t()), dict(weight=w.double()), dict(weight=w[:8]), dict(y=y[:3]), dict(h=h.float()),
                dict(x=x.half()), dict(codes=torch.empty_like(x), scale=w)):
        args = dict(x=x, residual=r, weight=w, eps=EPS, h=h, y=y)
        args.update(bad)
        with pytest.raises((ValueError, nat.MoEError)):
            nat.moe_rmsnorm(**args)


# dw of many rows.  A part of the launch takes every parts-th row, one multiply-add
# each; there is at least one part per SM (or per row), so ceil(T / SMs) roundings.
# Then 32 groups of the at most 1184 parts (more below 512 columns: 9472) in turn, and
# the groups: at most ceil(parts / 32) + 32.  n carries 2^-18.
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(6000, 64), (5000, 1032), (5000, 4104), (4100, 7168), (3000, 8200), (700, 32768)])
def test_weight_gradient_of_many_rows(cuda_device, T, d, dt):
    h, dy = (rows_of(T, d, dt, cuda_device, s) for s in (17, 18))
    w = 1.0 + 0.1 * torch.randn(d, device=cuda_device)
    dh, dw = backward(h, w, dy, None)
    want, wantw, size, sizew = ref.rmsnorm_backward(h.cpu(), w.cpu(), EPS, dy.cpu(), None)
    assert ((dh.cpu().double() - want).abs() <= want.abs() * HALF[dt] * (1 + 2.0 ** -16) + size * 2.0 ** -17).all()
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    parts = 1184 if d >= 512 else 9472
    adds = -(-T // sms) + -(-parts // 32) + 32
    assert ((dw.cpu().double() - wantw).abs() <= sizew * (adds * 2.0 ** -24 + FP32)).all()
