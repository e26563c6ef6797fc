"""Plain 64-bit implementations of the operators around the experts, on CPU
tensors: the RMS norm with residual and 8-bit output, the group-limited
routing, and the experts in e4m3 with one scale per block of 128.  Written from
the formulas, one row or expert at a time where that is clearest.
"""
import itertools
import math

import torch

F64 = torch.float64
LEAST = 2.0 ** -100


# ---------------------------------------------------------------- RMS norm
def rmsnorm(x, residual, weight, eps):
    """z and v in 64 bits."""
    z = x.to(F64) + (0.0 if residual is None else residual.to(F64))
    v = z / torch.sqrt((z * z).mean(1, keepdim=True) + eps) * weight.to(F64)
    return z, v


def rmsnorm_backward(h, weight, eps, dy, dres):
    """dh, dweight, and the magnitudes their roundings are relative to."""
    h, w, dy = h.to(F64), weight.to(F64), dy.to(F64)
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    n, u = h * rstd, dy * w
    mean = (u * n).mean(1, keepdim=True)
    res = torch.zeros_like(h) if dres is None else dres.to(F64)
    dh = res + rstd * (u - n * mean)
    size = res.abs() + rstd * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True))
    return dh, (dy * n).sum(0), size, (dy * n).abs().sum(0)


def block_max(v):
    """Largest magnitude of each run of 128 values of a row, at least 2^-100."""
    cols = [v[:, c:c + 128].abs().amax(1) for c in range(0, v.shape[1], 128)]
    return torch.stack(cols, 1).clamp(min=LEAST)


def spread(scale, width):
    """A row's block scales, one per column."""
    return scale.repeat_interleave(128, 1)[:, :width]


def quantize(v):
    """Codes' values and scales of 64-bit rows."""
    top = block_max(v)
    return (v * spread(448.0 / top, v.shape[1])).to(torch.float32).to(torch.float8_e4m3fn).to(F64), top / 448.0


# ---------------------------------------------------------------- routing
def scores(logits, score):
    l = logits.to(F64)
    if score == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m))
        z = e.sum(1, keepdim=True)
        return torch.where(z == 0, torch.zeros_like(e), e / z)
    return 1.0 / (1.0 + torch.exp(-l))


def _rank(v):                                       # NaN below every number
    return -math.inf if math.isnan(v) else v


def _choices(row, k, n_group, topk_group, group_top, tau):
    """The choice of one row of keys, by Python's own sort of (key, id); with
    tau > 0 every choice that group scores moved by at most tau / 2 can give."""
    E = len(row)
    size = E // n_group
    total = []
    for g in range(n_group):
        best = sorted((_rank(v) for v in row[g * size:(g + 1) * size]), reverse=True)[:group_top]
        total.append(_rank(sum(best)))
    order = sorted(range(n_group), key=lambda g: (-total[g], g))
    border = total[order[topk_group - 1]]
    if tau:
        sure = [g for g in order if total[g] > border + tau]
        near = [g for g in order if abs(total[g] - border) <= tau or total[g] == border]
        sets = [sure + list(c) for c in itertools.combinations(near, topk_group - len(sure))]
    else:
        sets = [order[:topk_group]]
    found = []
    for kept in sets:
        ids = [e for e in range(E) if e // size in kept]
        ids.sort(key=lambda e: (math.isnan(row[e]), -_rank(row[e]), e))
        found.append(ids[:k])
    return found


def _keys(logits, sel_bias, score):
    key = logits.to(F64) if score == "softmax" else scores(logits, score)
    return (key if sel_bias is None else key + sel_bias.to(F64)).tolist()


def select(logits, sel_bias, k, n_group, topk_group, group_top, score):
    return torch.tensor([_choices(r, k, n_group, topk_group, group_top, 0.0)[0]
                         for r in _keys(logits, sel_bias, score)], dtype=torch.int32)


def check_choice(idx, logits, sel_bias, k, n_group, topk_group, group_top, score):
    """idx is the choice, where 64-bit arithmetic decides it.  Sums of two keys
    can lie closer together than that: a sigmoid of two fp64 implementations is
    off by at most 3 roundings of 2^-53 (exp within an ulp, the sum, the
    quotient; s <= 1), a key with its bias (|key| < 2 here) by 2 more, so a
    score by 2 * 5 + 2 of them, and the difference of two scores by 24 * 2^-53.
    Groups within 2^-48 of the border may therefore fall on either side of it;
    keys themselves differ by far more or not at all, so nothing else moves."""
    want = select(logits, sel_bias, k, n_group, topk_group, group_top, score)
    keys = _keys(logits, sel_bias, score)
    for t in (idx != want).any(1).nonzero().flatten().tolist():
        assert group_top == 2 and idx[t].tolist() in _choices(keys[t], k, n_group, topk_group, group_top, 2.0 ** -48), \
            (t, idx[t].tolist(), want[t].tolist())


def gates(logits, idx, score, renorm, scale):
    g = scores(logits, score).gather(1, idx.long())
    if score == "sigmoid" or renorm:
        total = g.sum(1, keepdim=True)
        g = torch.where(total == 0, torch.zeros_like(g), g / total)
    return g * scale


def score_sums(logits, score):
    s = scores(logits, score)
    z = s.sum(1, keepdim=True)
    s = torch.where(z == 0, torch.zeros_like(s), s / z)
    return torch.stack([s[t:t + 32].sum(0) for t in range(0, s.shape[0], 32)])


def route_loss(logits, idx, dgate, counts, alpha, score, renorm, scale):
    """sum dgate * gate + alpha * E * sum f P: what the routing gradient is of."""
    T, E = logits.shape
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    g = s.gather(1, idx.long())
    if score == "sigmoid" or renorm:
        g = g / g.sum(1, keepdim=True)
    P = (s / s.sum(1, keepdim=True)).mean(0)
    f = counts.to(F64) / (T * idx.shape[1])
    return (dgate * g).sum() * scale + alpha * E * (f * P).sum()


def route_backward(logits, idx, dgate, counts, alpha, score, renorm, scale):
    l = logits.to(F64).requires_grad_(True)
    return torch.autograd.grad(route_loss(l, idx, dgate.to(F64), counts, alpha, score, renorm, scale), l)[0]


# ---------------------------------------------------------------- experts
def dequantize(codes, scale):
    """Rows of e4m3 codes (uint8) with a scale per 128 values."""
    nb = (codes.shape[1] + 127) // 128
    return codes.view(torch.float8_e4m3fn).to(F64) * spread(scale[:, :nb].to(F64), codes.shape[1])


def dequantize_weight(codes, scale):
    return dequantize(codes, scale.repeat_interleave(128, 0)[:codes.shape[0]])


def _product(x, w, blocks):
    """x w^T, and a bound on its fp32 error: sums of a block of 128 and then of
    the scaled blocks, every addition and scaling off by at most 2^-23 of the
    magnitudes it works on (the tensor core truncates)."""
    return x @ w.T, (x.abs() @ w.abs().T) * (blocks + 16) * 2.0 ** -23


def ffn(x, w1, wu, w2, b1, b2, far=False):
    """Output rows of one expert on dequantized rows x, and a bound on how far
    a computation with fp32 sums may be off before its last rounding.  A hidden
    value within its fp32 error of the middle between two codes may take either
    code: the bound adds that step times its weights.

    far: for arguments of the SiLU beyond 90 as well.  exp(-a) is 0 or infinite
    there, so the result is a, or 0 where the exact value is below 90 e^-90 |u|,
    and its error grows no further with |a|; and codes saturate at -448 as at 448."""
    blocks = (x.shape[1] + 127) // 128
    a, ea = _product(x, w1, blocks)
    if wu is None:
        if b1 is not None:
            a = a + b1.to(F64)
        h = 0.5 * a * (1.0 + torch.erf(a / math.sqrt(2.0)))
        eh = 1.13 * ea + a.abs() * 2.0 ** -20       # |gelu'| <= 1.13; erff and the products
    else:
        u, eu = _product(x, wu, blocks)
        s = a / (1.0 + torch.exp(-a))
        h = s * u
        eh = 1.1 * ea * u.abs() + s.abs() * eu + h.abs() * (10 + 1.5 * (a.abs().clamp(max=90.0) if far else a.abs())) * 2.0 ** -23
    width = h.shape[1]
    top = block_max(h)
    etop = block_max(eh)                            # the maximum moves by at most the largest error
    rel = spread(etop / top, width)
    q = h * spread(448.0 / top, width)
    eq = eh * spread(448.0 / top, width) + q.abs() * (rel + 2.0 ** -22)
    lo = (q - eq).clamp(min=-448.0 if far else -math.inf).to(torch.float32).to(torch.float8_e4m3fn).to(F64)
    hi = (q + eq).clamp(max=448.0).to(torch.float32).to(torch.float8_e4m3fn).to(F64)
    mid = q.to(torch.float32).to(torch.float8_e4m3fn).to(F64)
    flip = torch.maximum(hi - mid, mid - lo)
    scale = spread(top / 448.0, width)
    hd = mid * scale
    eh2 = flip * scale + hd.abs() * (rel + 2.0 ** -22)
    y, ey = _product(hd, w2, (width + 127) // 128)
    ey = ey + eh2 @ w2.abs().T
    if b2 is not None:
        y = y + b2.to(F64)
        ey = ey + y.abs() * 2.0 ** -23
    return y, ey
