"""The block around an MoE layer's experts, operator by operator: the RMS norm
with the residual's addition and an 8-bit output, the routing to experts in
groups, and the experts' products in e4m3 with one scale per block of 128.

Each case runs either the plain form (elementary torch operations in 32 bits,
in 64 where a comparison decides) or, with ``own`` set, the calls a program
makes of this package.
"""
import math

import torch

own = False

BLOCK = 128                     # values per scale
LEAST = 2.0 ** -100             # smallest block maximum a scale is made from
EPS = 1e-6


def listed():
    return [
        # one decoding step of four sequences: latency only
        dict(name="norm_decode", op="norm", T=4, d=2048, dtype="bf16", quant=True),
        # a prefill batch of the widest layer: pure memory traffic
        dict(name="norm_prefill", op="norm", T=8192, d=7168, dtype="bf16", quant=True),
        # the fp32 layer, a width that ends inside a block, no 8-bit output
        dict(name="norm_f32_odd", op="norm", T=3001, d=1160, dtype="f32", quant=False),
        # a training step's backward pass, with the gradient of the residual stream
        dict(name="norm_backward", op="norm_bwd", T=16384, d=2048, dtype="bf16"),
        # one decoding step of 16 sequences through 256 experts in 8 groups
        dict(name="route_decode", op="route", T=16, E=256, k=8, n_group=8, topk_group=4, group_top=2,
             score="sigmoid", renorm=1, bias=True, scale=2.5),
        # the same router on a prefill batch
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, n_group=8, topk_group=4, group_top=2,
             score="sigmoid", renorm=1, bias=True, scale=2.5),
        # a training step's router gradient, balance loss included
        dict(name="route_backward", op="route_bwd", T=16384, E=128, k=8, n_group=4, topk_group=2, group_top=1,
             score="softmax", renorm=1, bias=False, scale=1.0),
        # a single token: the weights of eight small experts stream by
        dict(name="experts_decode", op="experts", T=1, d=2048, E=128, F=768, k=8, act="swiglu", S=0, skew=0.0),
        # 64 tokens on one rank's 32 wide experts and the shared expert
        dict(name="experts_decode_wide", op="experts", T=64, d=7168, E=32, F=2048, k=8, act="swiglu", S=2048,
             skew=0.0),
        # prefill over many small experts with uneven popularity
        dict(name="experts_prefill", op="experts", T=16384, d=2048, E=128, F=768, k=8, act="swiglu", S=0, skew=1.1),
        # prefill over few large experts
        dict(name="experts_prefill_wide", op="experts", T=4096, d=4096, E=8, F=14336, k=2, act="swiglu", S=0,
             skew=0.0),
        # GELU experts with biases, widths that end inside a block, experts without rows
        dict(name="experts_gelu_ragged", op="experts", T=1000, d=1040, E=16, F=2064, k=2, act="gelu", S=0, skew=2.0),
    ]


def _log(rng, lo, hi, step=1):
    """A size in lo..hi, even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_bwd", "route", "route", "route_bwd", "experts", "experts", "experts"))
    if op in ("norm", "norm_bwd"):
        d = _log(rng, 64, 8192, 8)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        case = dict(op=op, T=_log(rng, 1, min(32768, 50_000_000 // d)), d=d, dtype=dtype)
        if op == "norm":
            case["quant"] = dtype == "bf16" or rng.random() < 0.3
        return case
    if op in ("route", "route_bwd"):
        n_group = rng.choice((1, 2, 4, 5, 8))
        size = rng.choice([s for s in (4, 6, 8, 12, 16, 20, 32, 64) if s * n_group <= 256])
        topk_group = rng.randint(1, n_group)
        return dict(op=op, T=_log(rng, 1, 16384), E=n_group * size, k=rng.randint(1, min(8, topk_group * size)),
                    n_group=n_group, topk_group=topk_group, group_top=rng.choice((1, 2)),
                    score=rng.choice(("softmax", "sigmoid")), renorm=rng.randint(0, 1), bias=rng.random() < 0.5,
                    scale=rng.choice((1.0, 2.5)))
    d, F = _log(rng, 256, 4096, 16), _log(rng, 256, 4096, 16)
    E = rng.choice((4, 8, 16, 32, 64))
    k = rng.choice((1, 2, 4, 8) if E >= 8 else (1, 2))
    top = max(1, min(8192, int(8e11 / (6.0 * d * F * k))))
    return dict(op=op, T=_log(rng, 1, top), d=d, E=E, F=F, k=k, act=rng.choice(("swiglu", "swiglu", "gelu")),
                S=rng.choice((0, 0, 512)), skew=rng.choice((0.0, 1.1, 2.0)))


# ---------------------------------------------------------------- inputs
def _blocks(n):
    return -(-n // BLOCK)


def _quantize(v):
    """Codes (e4m3) and scales of fp32 or fp64 rows, one scale per 128 values."""
    n, nb = v.shape[-1], _blocks(v.shape[-1])
    p = torch.nn.functional.pad(v, (0, nb * BLOCK - n)).unflatten(-1, (nb, BLOCK))
    amax = p.abs().amax(-1).clamp(min=LEAST)
    codes = (p * (448.0 / amax).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)[..., :n]
    return codes.contiguous(), amax / 448.0


def _strided(scale, sld):
    """Scale rows of sld bytes, zero behind the last block."""
    return torch.nn.functional.pad(scale, (0, sld // 4 - scale.shape[-1])).contiguous()


def _weight(g, dev, E, out, inp, sld):
    """Codes of N(0, 1) draws and scales around 1 / sqrt(inputs), [E, out / 128, sld / 4]."""
    codes = torch.empty((E, out, inp), dtype=torch.float8_e4m3fn, device=dev)
    for e in range(E):
        codes[e] = torch.randn((out, inp), generator=g, device=dev).to(torch.float8_e4m3fn)
    scale = (torch.rand((E, _blocks(out), _blocks(inp)), generator=g, device=dev) + 0.5) / math.sqrt(inp)
    return codes, _strided(scale, sld)


def _counts(g, dev, T, E, k, skew):
    """Rows of each expert: every token picks k experts of popularity rank^-skew."""
    rank = torch.randperm(E, generator=g, device=dev).to(torch.float32) + 1.0
    weight = rank.pow(-skew).log()
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=dev).clamp(1e-20, 1 - 1e-7)))
    idx = (weight + noise).topk(k, dim=1).indices
    return torch.bincount(idx.flatten(), minlength=E)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case=dict(case))
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        T, d = c["T"], c["d"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # a residual stream with a few loud channels, a branch output around 1
        loud = torch.ones(d, device=dev)
        loud[torch.randperm(d, generator=g, device=dev)[:max(1, d // 256)]] = 20.0
        stream = (torch.randn((T, d), generator=g, device=dev) * loud * 2.0).to(dt)
        s["weight"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=dev)
        if c["op"] == "norm":
            s["residual"] = stream
            s["x"] = torch.randn((T, d), generator=g, device=dev).to(dt)
        else:
            s["h"] = stream
            s["dy"] = torch.randn((T, d), generator=g, device=dev).to(dt)
            s["dres"] = torch.randn((T, d), generator=g, device=dev).to(dt)
    elif c["op"] in ("route", "route_bwd"):
        T, E = c["T"], c["E"]
        s["logits"] = torch.randn((T, E), generator=g, device=dev)
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=dev) if c["bias"] else None
        if c["op"] == "route_bwd":
            s["idx"] = _select(c, s["logits"], s["bias"])[0]
            s["dgate"] = torch.randn((T, c["k"]), generator=g, device=dev)
            s["counts"] = torch.bincount(s["idx"].flatten().long(), minlength=E).to(torch.int32)
            s["alpha"] = 0.01
    else:
        T, d, E, F, k, S = c["T"], c["d"], c["E"], c["F"], c["k"], c["S"]
        sld = -(-4 * _blocks(max(d, F, S)) // 16) * 16
        s["sld"] = sld
        counts = _counts(g, dev, T, E, k, c["skew"])
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        offsets[1:] = counts.cumsum(0)
        s["offsets"], s["rows"] = offsets, counts.tolist()
        rows = torch.randn((T * k, d), generator=g, device=dev)
        codes, scale = _quantize(rows)
        s["x8"], s["xs"] = codes, _strided(scale, sld)
        s["row_gate"] = torch.rand(T * k, generator=g, device=dev) * (2.0 / k)
        w = {}
        w["W1"], w["W1_scale"] = _weight(g, dev, E, F, d, sld)
        if c["act"] == "swiglu":
            w["Wu"], w["Wu_scale"] = _weight(g, dev, E, F, d, sld)
        w["W2"], w["W2_scale"] = _weight(g, dev, E, d, F, sld)
        s["b1"] = s["b2"] = s["xt8"] = s["xts"] = None
        if c["act"] == "gelu":
            s["b1"] = (torch.rand((E, F), generator=g, device=dev) - 0.5) * 0.02
            s["b2"] = (torch.rand((E, d), generator=g, device=dev) - 0.5) * 0.02
        if S:
            w["Wsg"], w["Wsg_scale"] = (t[0] for t in _weight(g, dev, 1, S, d, sld))
            if c["act"] == "swiglu":
                w["Wsu"], w["Wsu_scale"] = (t[0] for t in _weight(g, dev, 1, S, d, sld))
            w["Wsd"], w["Wsd_scale"] = (t[0] for t in _weight(g, dev, 1, d, S, sld))
            codes, scale = _quantize(torch.randn((T, d), generator=g, device=dev))
            s["xt8"], s["xts"] = codes, _strided(scale, sld)
        s["w"] = w
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program keeps between the calls: configuration, output buffers, workspaces."""
    from mixture_experts_layer_49_b200 import native as nat

    c, dev = s["case"], torch.device("cuda")
    if c["op"] == "norm":
        x, T, d = s["x"], c["T"], c["d"]
        s["h"], s["y"] = torch.empty_like(x), torch.empty_like(x)
        s["codes"] = torch.empty((T, d), dtype=torch.uint8, device=dev) if c["quant"] else None
        s["scale"] = torch.zeros((T, -(-_blocks(d) // 4) * 4), device=dev) if c["quant"] else None
    elif c["op"] == "norm_bwd":
        s["dh"], s["dweight"] = torch.empty_like(s["h"]), torch.empty_like(s["weight"])
        s["ws"] = nat.alloc_rmsnorm_backward_workspace(c["T"], c["d"])
    elif c["op"] in ("route", "route_bwd"):
        s["cfg"] = nat.make_config(c["T"], 8, c["E"], 8, c["k"], score=c["score"], renorm=c["renorm"])
        s["groups"] = nat.route_groups(c["n_group"], c["topk_group"], c["group_top"], c["scale"])
        if c["op"] == "route":
            s["idx"] = torch.empty((c["T"], c["k"]), dtype=torch.int32, device=dev)
            s["gate"] = torch.empty((c["T"], c["k"]), device=dev)
            s["psum"] = torch.empty((nat.router_blocks(s["cfg"]), c["E"]), device=dev)
        else:
            s["dlogits"] = torch.empty_like(s["logits"])
    else:
        s["cfg"] = nat.make_config(c["T"], c["d"], c["E"], c["F"], c["k"], act=c["act"], d_ff_shared=c["S"])
        s["experts"] = nat.fp8_block_experts(s["w"], s["sld"])
        s["ws"] = nat.alloc_workspace(s["cfg"])
        s["y"] = torch.empty((nat.perm_rows(s["cfg"]), c["d"]), dtype=torch.bfloat16, device=dev)


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _own_norm(s):
    from mixture_experts_layer_49_b200 import native as nat

    nat.moe_rmsnorm(s["x"], s["residual"], s["weight"], EPS, s["h"], s["y"], s["codes"], s["scale"])
    out = dict(h=s["h"], y=s["y"])
    if s["codes"] is not None:
        out["codes"] = s["codes"].view(torch.float8_e4m3fn)
        out["scale"] = s["scale"][:, :_blocks(s["case"]["d"])]
    return out


def _own_norm_bwd(s):
    from mixture_experts_layer_49_b200 import native as nat

    nat.moe_rmsnorm_backward(s["h"], s["weight"], EPS, s["dy"], s["dres"], s["dh"], s["dweight"], s["ws"])
    return dict(dh=s["dh"], dweight=s["dweight"])


def _own_route(s):
    from mixture_experts_layer_49_b200 import native as nat

    nat.moe_route_select(s["cfg"], s["groups"], s["logits"], s["bias"], s["idx"], s["gate"], s["psum"])
    return dict(idx=s["idx"], gate=s["gate"], psum=s["psum"])


def _own_route_bwd(s):
    from mixture_experts_layer_49_b200 import native as nat

    nat.moe_route_backward(s["cfg"], s["groups"], s["logits"], s["idx"], s["dgate"], s["counts"], s["alpha"],
                           s["dlogits"])
    return dict(dlogits=s["dlogits"])


def _own_experts(s):
    from mixture_experts_layer_49_b200 import native as nat

    nat.moe_grouped_ffn_fp8_block(s["cfg"], s["x8"], s["xs"], s["offsets"], s["row_gate"], s["experts"], s["b1"],
                                  s["b2"], s["xt8"], s["xts"], s["y"], s["ws"])
    return dict(y=s["y"])


def _plain_norm(s):
    z = s["x"].float() + s["residual"].float()
    v = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["weight"]
    out = dict(h=z.to(s["x"].dtype), y=v.to(s["x"].dtype))
    if s["case"]["quant"]:
        out["codes"], out["scale"] = _quantize(v)
    return out


def _plain_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, u = h * rstd, dy * s["weight"]
    dh = s["dres"].float() + rstd * (u - n * (u * n).mean(-1, keepdim=True))
    return dict(dh=dh.to(s["h"].dtype), dweight=(dy * n).sum(0))


def _scores(c, logits):
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        return e / e.sum(-1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-logits))


def _select(c, logits, bias):
    """The chosen experts (int32) and the selection keys, in 64 bits: neighbours in
    rank may lie closer together than 32 bits tell."""
    T, E, G = logits.shape[0], c["E"], c["n_group"]
    key = logits.double() if c["score"] == "softmax" else _scores(c, logits.double())
    if bias is not None:
        key = key + bias.double()
    by_group = key.view(T, G, E // G)
    top = by_group.sort(dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
    kept = top.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
    out = torch.ones((T, G), dtype=torch.bool, device=key.device).scatter_(1, kept, False)
    masked = by_group.masked_fill(out.unsqueeze(-1), -math.inf).view(T, E)
    return masked.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]].to(torch.int32), key


def _plain_route(s):
    c = s["case"]
    idx, _ = _select(c, s["logits"], s["bias"])
    score = _scores(c, s["logits"])
    gate = score.gather(1, idx.long())
    if c["score"] == "sigmoid" or c["renorm"]:
        gate = gate / gate.sum(-1, keepdim=True)
    share = score if c["score"] == "softmax" else score / score.sum(-1, keepdim=True)
    T, E = share.shape
    share = torch.nn.functional.pad(share, (0, 0, 0, -T % 32))
    return dict(idx=idx, gate=gate * c["scale"], psum=share.view(-1, 32, E).sum(1))


def _plain_route_bwd(s):
    c, score, idx = s["case"], _scores(s["case"], s["logits"]), s["idx"].long()
    T, E = score.shape
    dg = s["dgate"] * c["scale"]
    chosen = score.gather(1, idx)
    if c["score"] == "sigmoid" or c["renorm"]:
        total = chosen.sum(-1, keepdim=True)
        dg = (dg - (dg * chosen).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(score).scatter_(1, idx, dg)
    f = s["counts"].float() / (T * c["k"])
    dshare = (s["alpha"] * E / T) * f
    if c["score"] == "softmax":
        ds = ds + dshare
        return dict(dlogits=score * (ds - (ds * score).sum(-1, keepdim=True)))
    total = score.sum(-1, keepdim=True)
    ds = ds + (dshare - (score * dshare).sum(-1, keepdim=True) / total) / total
    return dict(dlogits=ds * score * (1.0 - score))


def _dequantize(codes, scale, dtype):
    """Rows of codes with one scale per 128 values of the row."""
    spread = scale[..., :_blocks(codes.shape[-1])].to(dtype).repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]
    return codes.to(dtype) * spread


def _dequantize_weight(codes, scale, dtype):
    return _dequantize(codes, scale.repeat_interleave(BLOCK, 0)[:codes.shape[0]], dtype)


def _plain_ffn(x, w1, wu, w2, b1, b2):
    a = x @ w1.T
    if wu is None:
        a = a if b1 is None else a + b1
        hidden = 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))
    else:
        hidden = a / (1.0 + torch.exp(-a)) * (x @ wu.T)
    y = _dequantize(*_quantize(hidden), torch.float32) @ w2.T
    return y if b2 is None else y + b2


def _plain_experts(s):
    c, w, f32 = s["case"], s["w"], torch.float32
    swiglu = c["act"] == "swiglu"
    rows = c["T"] * c["k"]
    y = torch.empty((rows + (c["T"] if c["S"] else 0), c["d"]), dtype=torch.bfloat16, device=s["x8"].device)
    at = 0
    for e, n in enumerate(s["rows"]):              # each expert has its own number of rows
        if n == 0:
            continue
        part = slice(at, at + n)
        at += n
        m = [_dequantize_weight(w[k][e], w[k + "_scale"][e], f32) if k in w else None for k in ("W1", "Wu", "W2")]
        out = _plain_ffn(_dequantize(s["x8"][part], s["xs"][part], f32), *m,
                         None if swiglu else s["b1"][e], None if swiglu else s["b2"][e])
        y[part] = (out * s["row_gate"][part].unsqueeze(1)).to(torch.bfloat16)
    if c["S"]:
        m = [_dequantize_weight(w[k], w[k + "_scale"], f32) if k in w else None for k in ("Wsg", "Wsu", "Wsd")]
        y[rows:] = _plain_ffn(_dequantize(s["xt8"], s["xts"], f32), *m, None, None).to(torch.bfloat16)
    return dict(y=y)


_own = dict(norm=_own_norm, norm_bwd=_own_norm_bwd, route=_own_route, route_bwd=_own_route_bwd, experts=_own_experts)
_plain = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, route=_plain_route, route_bwd=_plain_route_bwd,
              experts=_plain_experts)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        n, b = c["T"] * c["d"], 2 if c["dtype"] == "bf16" else 4
        quant = n + c["T"] * 4 * _blocks(c["d"]) if c["quant"] else 0
        return dict(bytes=4 * n * b + quant + 4 * c["d"], flops=8 * n)
    if c["op"] == "norm_bwd":
        n, b = c["T"] * c["d"], 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=4 * n * b + 8 * c["d"], flops=14 * n)
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=4 * T * E + 8 * T * k + 4 * E * (-(-T // 32)), flops=8 * T * E)
    if c["op"] == "route_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=8 * T * E + 8 * T * k, flops=12 * T * E)
    T, d, E, F, k, S = c["T"], c["d"], c["E"], c["F"], c["k"], c["S"]
    mats = 3 if c["act"] == "swiglu" else 2
    hit = E * (1.0 - (1.0 - 1.0 / E) ** (T * k)) if T > 1 else min(E, k)     # experts that get a row
    rows = T * k
    by = hit * mats * d * F * (1 + 4 / BLOCK ** 2) + rows * (d * (1 + 4 / BLOCK) + 4 + 2 * d)
    if S:
        by += mats * d * S * (1 + 4 / BLOCK ** 2) + T * (d * (1 + 4 / BLOCK) + 2 * d)
    return dict(bytes=by, flops=2.0 * mats * d * (rows * F + T * S))


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    c = case
    if c["op"] == "norm":
        z = s["x"].to(f64) + s["residual"].to(f64)
        v = s["weight"].to(f64) * z / (z.pow(2).sum(1, keepdim=True) / c["d"] + EPS).sqrt()
        out = dict(h=z, y=v)
        if c["quant"]:
            nb = _blocks(c["d"])
            room = torch.zeros((c["T"], nb * BLOCK), dtype=f64, device=v.device)
            room[:, :c["d"]] = v
            most = room.view(-1, nb, BLOCK).abs().max(-1).values.clamp(min=LEAST)
            # an 8-bit value stands for this one, before its rounding
            out["codes"] = (room.view(-1, nb, BLOCK) / most[..., None] * 448.0).view(c["T"], -1)[:, :c["d"]]
            out["scale"] = most / 448.0
        return out
    if c["op"] == "norm_bwd":
        h, dy, w = s["h"].to(f64), s["dy"].to(f64), s["weight"].to(f64)
        q = h.pow(2).sum(1, keepdim=True) / c["d"] + EPS
        inner = (dy * w * h).sum(1, keepdim=True) / c["d"]
        return dict(dh=s["dres"].to(f64) + dy * w / q.sqrt() - h * inner / q.pow(1.5),
                    dweight=torch.einsum("td,td->d", dy, h / q.sqrt()))
    if c["op"] in ("route", "route_bwd"):
        l = s["logits"].to(f64)
        p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        share = p / p.sum(1, keepdim=True)
        divided = c["score"] == "sigmoid" or c["renorm"] == 1
        if c["op"] == "route":
            idx = _select(c, s["logits"], s["bias"])[0].long()
            g = torch.take_along_dim(p, idx, 1)
            if divided:
                g = g / g.sum(1, keepdim=True)
            block = torch.arange(c["T"], device=l.device) // 32
            psum = torch.zeros((-(-c["T"] // 32), c["E"]), dtype=f64, device=l.device).index_add_(0, block, share)
            return dict(idx=None, gate=g * c["scale"], psum=psum)
        idx, dgate = s["idx"].long(), s["dgate"].to(f64) * c["scale"]
        f = s["counts"].to(f64) / (c["T"] * c["k"])
        l = l.detach().requires_grad_(True)
        p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        g = torch.take_along_dim(p, idx, 1)
        if divided:
            g = g / g.sum(1, keepdim=True)
        mean = (p / p.sum(1, keepdim=True)).mean(0)
        loss = (g * dgate).sum() + s["alpha"] * c["E"] * (f * mean).sum()
        return dict(dlogits=torch.autograd.grad(loss, l)[0])
    w, T, k, d = s["w"], c["T"], c["k"], c["d"]

    def wide(codes, scale):
        n, m = codes.shape
        i = torch.arange(n, device=codes.device) // BLOCK
        j = torch.arange(m, device=codes.device) // BLOCK
        return codes.to(f64) * scale.to(f64)[i][:, j]

    def expert(x8, xs, get, b1, b2):
        j = torch.arange(d, device=x8.device) // BLOCK
        x = x8.to(f64) * xs.to(f64)[:, j]
        a = x @ get("1").T
        if c["act"] == "swiglu":
            hid = torch.nn.functional.silu(a) * (x @ get("u").T)
        else:
            hid = torch.nn.functional.gelu(a if b1 is None else a + b1.to(f64))
        width = hid.shape[1]
        for lo in range(0, width, BLOCK):                 # the hidden row in 8 bits, block by block
            part = hid[:, lo:lo + BLOCK]
            most = part.abs().max(1, keepdim=True).values.clamp(min=LEAST)
            hid[:, lo:lo + BLOCK] = (part / most * 448.0).to(torch.float8_e4m3fn).to(f64) * (most / 448.0)
        y = hid @ get("2").T
        return y if b2 is None else y + b2.to(f64)

    y = torch.zeros((T * k + (T if c["S"] else 0), d), dtype=f64, device=s["x8"].device)
    at = 0
    for e, n in enumerate(s["rows"]):
        if n:
            name = {"1": "W1", "u": "Wu", "2": "W2"}
            b1, b2 = (None, None) if s["b1"] is None else (s["b1"][e], s["b2"][e])
            out = expert(s["x8"][at:at + n], s["xs"][at:at + n],
                         lambda m: wide(w[name[m]][e], w[name[m] + "_scale"][e]), b1, b2)
            y[at:at + n] = out * s["row_gate"][at:at + n].to(f64)[:, None]
            at += n
    if c["S"]:
        name = {"1": "Wsg", "u": "Wsu", "2": "Wsd"}
        y[T * k:] = expert(s["xt8"], s["xts"], lambda m: wide(w[name[m]], w[name[m] + "_scale"]), None, None)
    return dict(y=y)
