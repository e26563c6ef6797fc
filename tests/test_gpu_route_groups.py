"""Group-limited routing against a 64-bit sort, row by row, and its gradient.

Tolerances.  The choice is that of the 64-bit keys (block_reference.check_choice
says what 64-bit arithmetic leaves open).  Gates
and score sums: expf within 2 ulp on an argument that one subtraction rounded
(|l - m| <= 32 here: 32 * 2^-24), a sum of at most 8 + 5 terms a warp, a
reciprocal or quotient and three products: at most 2^-17.7 relative with the
sum over 32 tokens; 2^-17 is used.  The gradient: the same relative error on
each term that meets, twice (scores and normalisation): 2^-15 of the magnitudes.
"""
import pytest
import torch

from mixture_experts_layer_49_b200 import native as nat

import block_reference as ref

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -17


def config(T, E, k, score, renorm):
    return nat.make_config(T, 8, E, 8, k, score=score, renorm=renorm)


def run(logits, bias, k, groups, score="sigmoid", renorm=1):
    T, E = logits.shape
    cfg = config(T, E, k, score, renorm)
    idx = torch.full((T + 1, k), -9, dtype=torch.int32, device=logits.device)
    gate = torch.full((T + 1, k), -9.0, device=logits.device)
    psum = torch.full(((T + 31) // 32 + 1, E), -9.0, device=logits.device)
    nat.moe_route_select(cfg, nat.route_groups(*groups), logits, bias, idx, gate, psum)
    assert (idx[T] == -9).all() and (gate[T] == -9).all() and (psum[-1] == -9).all()
    return idx[:T], gate[:T], psum[:-1]


def check(logits, bias, k, groups, score="sigmoid", renorm=1):
    idx, gate, psum = run(logits, bias, k, groups, score, renorm)
    l, b = logits.cpu(), None if bias is None else bias.cpu()
    ref.check_choice(idx.cpu(), l, b, k, *groups[:3], score)
    g = ref.gates(l, idx.cpu(), score, renorm, groups[3])
    assert ((gate.cpu().double() - g).abs() <= g.abs() * TOL + 1e-37).all()
    p = ref.score_sums(l, score)
    assert ((psum.cpu().double() - p).abs() <= p.abs() * TOL + 1e-37).all()


CASES = [
    # E, k, groups
    (256, 8, (8, 4, 2, 2.5)), (256, 8, (8, 4, 1, 1.0)), (256, 32, (4, 2, 2, 1.0)), (256, 1, (32, 1, 2, 1.0)),
    (256, 6, (128, 5, 2, 1.0)), (256, 6, (256, 9, 1, 1.0)), (160, 6, (8, 3, 2, 16.0)), (128, 8, (4, 2, 2, 1.0)),
    (128, 8, (1, 1, 1, 1.0)), (64, 4, (16, 3, 2, 1.0)), (60, 4, (5, 2, 2, 1.0)), (30, 5, (5, 3, 2, 1.0)),
    (33, 3, (3, 2, 1, 1.0)), (32, 1, (8, 8, 2, 1.0)), (8, 2, (4, 2, 2, 1.0)), (7, 7, (1, 1, 2, 1.0)),
    (250, 8, (25, 7, 2, 1.0)), (1, 1, (1, 1, 1, 2.0)),
]


@pytest.mark.parametrize("score,renorm,bias", [("sigmoid", 1, True), ("sigmoid", 0, False), ("softmax", 1, True),
                                               ("softmax", 0, False)])
@pytest.mark.parametrize("E,k,groups", CASES)
def test_selection(cuda_device, E, k, groups, score, renorm, bias):
    g = torch.Generator(device=cuda_device).manual_seed(E * 100 + k)
    for T in (1, 45, 64):
        logits = 2.0 * torch.randn((T, E), generator=g, device=cuda_device)
        b = 0.3 * torch.randn(E, generator=g, device=cuda_device) if bias else None
        check(logits, b, k, groups, score, renorm)


@pytest.mark.parametrize("score,renorm,bias", [("sigmoid", 1, True), ("softmax", 0, False)])
@pytest.mark.parametrize("E,k,groups", CASES)
def test_many_tokens(cuda_device, E, k, groups, score, renorm, bias):
    """More blocks than SMs take four tokens to a warp: the same choices as in
    calls of few tokens, gates and sums each within TOL of the exact ones."""
    g = torch.Generator(device=cuda_device).manual_seed(E * 100 + k + 1)
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    T = 32 * (sms + 9) + 5
    logits = 2.0 * torch.randn((T, E), generator=g, device=cuda_device)
    b = 0.3 * torch.randn(E, generator=g, device=cuda_device) if bias else None
    idx, gate, psum = run(logits, b, k, groups, score, renorm)
    for t in range(0, T, 1024):
        i, w, p = run(logits[t:t + 1024], b, k, groups, score, renorm)
        assert torch.equal(idx[t:t + 1024], i)
        assert ((gate[t:t + 1024] - w).abs() <= 2 * TOL * w.abs() + 2e-37).all()
        q = psum[t // 32:t // 32 + p.shape[0]]
        assert ((q - p).abs() <= 2 * TOL * p.abs() + 2e-37).all()


def test_unaligned_rows(cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(4)
    raw = torch.randn(64 * 256 + 3, generator=g, device=cuda_device)
    for off in (0, 1, 3):
        logits = raw[off:off + 64 * 256].view(64, 256)
        check(logits, None, 8, (8, 4, 2, 2.5))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_close_keys_are_told_apart(cuda_device, score):
    """Logits a few units in the last place apart, and in saturated sigmoids: fp32
    keys would tie or swap, the 64-bit values do not."""
    T, E = 256, 64
    g = torch.Generator(device=cuda_device).manual_seed(11)
    base = torch.randn((T, 1), generator=g, device=cuda_device)
    ulps = torch.randint(-6, 7, (T, E), generator=g, device=cuda_device)
    logits = (base.view(torch.int32) + ulps.to(torch.int32)).view(torch.float32)
    logits[64:128] = 12.0 + torch.randn((64, E), generator=g, device=cuda_device)        # sigmoids near 1
    logits[128:160] = torch.randint(-3, 4, (32, E), generator=g, device=cuda_device).float()   # many exact ties
    bias = 1e-7 * torch.randn(E, generator=g, device=cuda_device)
    for b in (None, bias):
        for groups in ((1, 1, 1, 1.0), (8, 3, 2, 1.0), (4, 2, 1, 1.0)):
            check(logits.contiguous(), b, 6, groups, score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_take_the_lowest_ids(cuda_device, score):
    idx, _, _ = run(torch.zeros((3, 32), device=cuda_device), None, 4, (4, 2, 2, 1.0), score)
    assert (idx.cpu() == torch.arange(4, dtype=torch.int32)).all()
    logits = torch.zeros((1, 32), device=cuda_device)
    logits[0, ::2] = -0.0                                       # the same key
    assert run(logits, None, 4, (4, 2, 2, 1.0), score)[0].tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("score,renorm", [("sigmoid", 1), ("softmax", 1), ("softmax", 0)])
def test_masked_and_non_finite_logits(cuda_device, score, renorm):
    inf, nan = float("inf"), float("nan")
    logits = torch.randn((40, 64), device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(2))
    logits[0] = -inf                                            # nothing left
    logits[1, 3:] = -inf                                        # fewer experts left than are chosen
    logits[2, 16:32] = -inf                                     # a whole group masked
    logits[3] = torch.finfo(torch.float32).min
    logits[4, ::2] = torch.finfo(torch.float32).min
    logits[5, 17:] = -inf
    groups = (8, 3, 2, 2.0)
    check(logits, None, 4, groups, score, renorm)
    idx, gate, psum = run(logits, None, 4, groups, score, renorm)
    assert (gate[0] == 0).all() and idx[0].tolist() == [0, 1, 2, 3]
    logits[6, 5] = nan
    logits[7] = nan
    logits[8, 9] = inf
    logits[9, 8:16] = nan
    idx2, gate2, _ = run(logits, None, 4, groups, score, renorm)
    assert torch.equal(idx2[10:], idx[10:]) and torch.equal(gate2[10:], gate[10:])      # other rows as before
    assert torch.equal(idx2[:6], idx[:6]) and torch.equal(gate2[:6], gate[:6])
    assert torch.equal(idx2.cpu(), ref.select(logits.cpu(), None, 4, *groups[:3], score))
    for row in idx2.tolist():
        assert len(set(row)) == 4 and all(0 <= e < 64 for e in row)


def test_extreme_bias_and_no_psum(cuda_device):
    logits = torch.randn((70, 128), device=cuda_device)
    bias = torch.zeros(128, device=cuda_device)
    bias[7] = 1e30
    bias[9] = -1e30
    bias[40] = float("-inf")
    for score in ("sigmoid", "softmax"):
        check(logits, bias, 5, (4, 2, 2, 1.0), score)
    cfg = config(70, 128, 5, "softmax", 1)
    idx, gate = torch.empty((70, 5), dtype=torch.int32, device=cuda_device), torch.empty((70, 5), device=cuda_device)
    nat.moe_route_select(cfg, nat.route_groups(4, 2), logits, bias, idx, gate)
    assert torch.equal(idx.cpu(), ref.select(logits.cpu(), bias.cpu(), 5, 4, 2, 2, "softmax"))


@pytest.mark.parametrize("score,renorm", [("sigmoid", 1), ("softmax", 1), ("softmax", 0)])
@pytest.mark.parametrize("T,E,k,scale,alpha", [(1, 8, 1, 1.0, 0.0), (5, 256, 8, 2.5, 0.01), (70, 128, 8, 1.0, 1.0),
                                               (33, 60, 4, 2.5, 0.5), (64, 33, 32, 1.0, 0.0), (9, 1, 1, 1.0, 1.0)])
def test_gradient(cuda_device, T, E, k, scale, alpha, score, renorm):
    g = torch.Generator(device=cuda_device).manual_seed(T + E)
    logits = 2.0 * torch.randn((T, E), generator=g, device=cuda_device)
    idx = ref.select(logits.cpu(), None, k, 1, 1, 1, score).to(cuda_device)
    dgate = torch.randn((T, k), generator=g, device=cuda_device)
    counts = torch.bincount(idx.flatten().long(), minlength=E).to(torch.int32)
    cfg = config(T, E, k, score, renorm)
    d = torch.full((T + 1, E), -9.0, device=cuda_device)
    nat.moe_route_backward(cfg, nat.route_groups(1, 1, 1, scale), logits, idx, dgate, counts if alpha else None, alpha,
                           d[:T])
    assert (d[T] == -9).all()
    args = (idx.cpu(), dgate.cpu(), counts.cpu(), alpha, score, renorm, scale)
    want = ref.route_backward(logits.cpu(), *args)
    s = ref.scores(logits.cpu(), score)
    chosen = s.gather(1, idx.cpu().long())
    total = chosen.sum(1, keepdim=True) if (score == "sigmoid" or renorm) else 1.0
    # the magnitudes that meet: each score times the gradients it is weighed against
    own = torch.zeros_like(s).scatter_add_(1, idx.cpu().long(), dgate.cpu().double().abs() * scale / total)
    mean = (own * s).sum(1, keepdim=True)
    bal = alpha * E / T * counts.cpu().double() / (T * k)
    if score == "sigmoid":
        z = s.sum(1, keepdim=True)
        hit = torch.zeros_like(s).scatter_(1, idx.cpu().long(), 1.0)
        size = s * (1 - s) * (own + hit * mean / total + (bal + (bal * s).sum(1, keepdim=True) / z) / z)
    else:
        size = s * (own + 2 * mean + bal + (bal * s).sum(1, keepdim=True))
    assert ((d[:T].cpu().double() - want).abs() <= size * 2.0 ** -15 + 1e-37).all()


def test_gradient_of_bad_and_masked_rows(cuda_device):
    E, k = 64, 4
    logits = torch.randn((6, E), device=cuda_device)
    logits[1] = float("-inf")
    logits[2, 8:] = float("-inf")
    idx = torch.arange(k, dtype=torch.int32, device=cuda_device).repeat(6, 1).contiguous()
    idx[3, 1] = -1
    idx[4, 2] = E
    dgate = torch.randn((6, k), device=cuda_device)
    for score, renorm in (("sigmoid", 1), ("softmax", 1), ("softmax", 0)):
        d = torch.empty((6, E), device=cuda_device)
        nat.moe_route_backward(config(6, E, k, score, renorm), nat.route_groups(1, 1, 1), logits, idx, dgate, None, 0.0, d)
        assert torch.isfinite(d).all() and (d[1] == 0).all() and (d[2, 8:] == 0).all()
        ok = ref.route_backward(logits[:1].cpu(), idx[:1].cpu(), dgate[:1].cpu(), torch.zeros(E), 0.0, score, renorm, 1.0)
        assert (d[0].cpu().double() - ok[0]).abs().max() < 1e-5


def test_two_calls_in_a_graph(cuda_device):
    T, E, k = 96, 256, 8
    a, b = torch.randn((T, E), device=cuda_device), torch.randn((T, E), device=cuda_device)
    cfg, groups = config(T, E, k, "sigmoid", 1), nat.route_groups(8, 4, 2, 2.5)
    outs = [(torch.empty((T, k), dtype=torch.int32, device=cuda_device), torch.empty((T, k), device=cuda_device),
             torch.empty((T // 32, E), device=cuda_device)) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for l, o in zip((a, b), outs):
            nat.moe_route_select(cfg, groups, l, None, *o)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for l, o in zip((a, b), outs):
        want = run(l, None, k, (8, 4, 2, 2.5))
        assert all(torch.equal(x, y) for x, y in zip(o, want))


def test_router_stage_agrees_with_the_selection_of_its_logits(cuda_device):
    """moe_router_topk_groups on x: its logits_out selected again give its outputs."""
    for dtype, T, d, E in (("bf16", 70, 256, 64), ("bf16", 1, 4096, 256), ("f32", 45, 128, 32)):
        g = torch.Generator(device=cuda_device).manual_seed(d)
        cfg = nat.make_config(T, d, E, 64, 4, dtype=dtype, score="sigmoid")
        x = torch.randn((T, d), generator=g, device=cuda_device).to(nat.layer_dtype(cfg))
        Wr = torch.randn((d, E), generator=g, device=cuda_device) / d ** 0.5
        lb, sb = (0.1 * torch.randn(E, generator=g, device=cuda_device) for _ in range(2))
        ws = nat.alloc_workspace(cfg)
        idx, gate = torch.empty((T, 4), dtype=torch.int32, device=cuda_device), torch.empty((T, 4), device=cuda_device)
        logits, psum = torch.empty((T, E), device=cuda_device), torch.empty((nat.router_blocks(cfg), E), device=cuda_device)
        groups = nat.route_groups(8, 3, 2, 1.5)
        nat.moe_router_topk_groups(cfg, groups, x, Wr, lb, sb, idx, gate, logits, psum, ws)
        plain = [torch.empty_like(t) for t in (idx, gate, logits, psum)]
        nat.moe_router_topk(cfg, x, Wr, lb, sb, *plain, ws)
        assert torch.equal(plain[2], logits)
        i2, g2, p2 = torch.empty_like(idx), torch.empty_like(gate), torch.empty_like(psum)
        nat.moe_route_select(cfg, groups, logits, sb, i2, g2, p2)
        assert torch.equal(i2, idx) and torch.equal(g2, gate) and torch.equal(p2, psum)
        nat.moe_router_topk_groups(cfg, groups, x, Wr, lb, sb, i2, g2, None, p2, ws)     # no logits asked for
        assert torch.equal(i2, idx) and torch.equal(g2, gate) and torch.equal(p2, psum)
        # one group: the same experts as the plain router
        nat.moe_router_topk_groups(cfg, nat.route_groups(1, 1, 1), x, Wr, lb, sb, i2, g2, None, p2, ws)
        want = ref.select(logits.cpu(), sb.cpu(), 4, 1, 1, 1, "sigmoid")
        assert torch.equal(i2.cpu(), want)
        assert nat.moe_get_device_status(ws) == nat.MOE_OK


@pytest.mark.parametrize("score,renorm", [("sigmoid", 1), ("softmax", 1), ("softmax", 0)])
@pytest.mark.parametrize("equal", [True, False])
def test_gradient_of_an_id_that_stands_twice(cuda_device, equal, score, renorm):
    """The slots of one id add up, whether their gate gradients are equal or not.
    dgate and logits are bounded by 1, k = 6: every term is at most 2.5 and a
    row adds fewer than 32 of them with 2^-15 each (the module's tolerance)."""
    T, E, k, scale, alpha = 40, 64, 6, 2.5, 0.5
    g = torch.Generator(device=cuda_device).manual_seed(21)
    logits = 2.0 * torch.rand((T, E), generator=g, device=cuda_device) - 1.0
    idx = torch.randint(0, 9, (T, k), generator=g, device=cuda_device).to(torch.int32)
    idx[0] = 5                                                  # one expert in every slot
    dgate = 2.0 * torch.rand((T, E if equal else k), generator=g, device=cuda_device) - 1.0
    if equal:                                                   # one gradient per expert
        dgate = dgate.gather(1, idx.long()).contiguous()
    counts = torch.bincount(idx.flatten().long(), minlength=E).to(torch.int32)
    d = torch.empty((T, E), device=cuda_device)
    nat.moe_route_backward(config(T, E, k, score, renorm), nat.route_groups(1, 1, 1, scale), logits, idx, dgate, counts,
                           alpha, d)
    want = ref.route_backward(logits.cpu(), idx.cpu(), dgate.cpu(), counts.cpu(), alpha, score, renorm, scale)
    assert ((d.cpu().double() - want).abs() <= 32 * 2.5 * 2.0 ** -15).all()


@pytest.mark.parametrize("lo,hi", [(-88.7, -87.0), (-88.7, -60.0), (-60.0, -50.0), (-30.0, -20.0), (-16.0, -8.0), (-8.0, 0.0),
                                   (0.0, 20.0), (-88.7, 3.0)])
def test_sigmoid_scores_of_any_size(cuda_device, lo, hi):
    """In units of 2^-24.  A score: expf 4 (2 ulp), sum 1, reciprocal 2 (1 ulp), a
    subnormal one (above 2^-128) 4 more: 11.  A gate: 11, the sum's 11 and 5
    shuffles, quotient and factor: 29 < 32.  A score sum: 11, the sum's 11 and 13
    additions, reciprocal and product, 32 tokens: 69 < 128."""
    g = torch.Generator(device=cuda_device).manual_seed(31)
    for E, groups in ((256, (8, 4, 2, 2.5)), (60, (5, 2, 1, 1.0))):
        logits = lo + (hi - lo) * torch.rand((64, E), generator=g, device=cuda_device)
        idx, gate, psum = run(logits, None, 8, groups)
        ref.check_choice(idx.cpu(), logits.cpu(), None, 8, *groups[:3], "sigmoid")
        want = ref.gates(logits.cpu(), idx.cpu(), "sigmoid", 1, groups[3])
        assert ((gate.cpu().double() - want).abs() <= want * 2.0 ** -19).all()
        want = ref.score_sums(logits.cpu(), "sigmoid")
        assert ((psum.cpu().double() - want).abs() <= want * 2.0 ** -17 + 1e-37).all()


@pytest.mark.parametrize("alpha", [0.0, 0.5])
def test_gradient_of_tiny_sigmoids(cuda_device, alpha):
    """Rows whose sigmoids are all tiny, and rows whose chosen ones are tiny beside
    the others': the same bound as test_gradient (scores below 2^-126 lose
    2^-22 of their value, within it).  Below -88.72 the fp32 score is 0: such rows'
    gradients are finite, and 0 where nothing chosen is left and alpha is 0."""
    T, E, k, scale = 64, 256, 8, 16.0
    g = torch.Generator(device=cuda_device).manual_seed(41)
    cfg, groups = config(T, E, k, "sigmoid", 1), nat.route_groups(1, 1, 1, scale)
    dgate = torch.randn((T, k), generator=g, device=cuda_device)
    d = torch.empty((T, E), device=cuda_device)

    def backward(logits, idx):
        counts = torch.bincount(idx.flatten().long(), minlength=E).to(torch.int32)
        nat.moe_route_backward(cfg, groups, logits, idx, dgate, counts if alpha else None, alpha, d)
        return counts.cpu()

    low = -88.7 + 0.4 * torch.rand((T, E), generator=g, device=cuda_device)
    wide = -88.7 + 30.0 * torch.rand((T, E), generator=g, device=cuda_device)
    mixed = 3.0 * torch.randn((T, E), generator=g, device=cuda_device)
    mixed[:, 128:] = low[:, 128:]
    for logits in (low, wide, mixed):
        idx = 128 + torch.rand((T, 128), generator=g, device=cuda_device).topk(k, 1).indices.to(torch.int32)
        counts = backward(logits, idx)
        want = ref.route_backward(logits.cpu(), idx.cpu(), dgate.cpu(), counts, alpha, "sigmoid", 1, scale)
        s = ref.scores(logits.cpu(), "sigmoid")
        total = s.gather(1, idx.cpu().long()).sum(1, keepdim=True)
        own = torch.zeros_like(s).scatter_add_(1, idx.cpu().long(), dgate.cpu().double().abs() * scale / total)
        mean = (own * s).sum(1, keepdim=True)
        bal = alpha * E / T * counts.double() / (T * k)
        z = s.sum(1, keepdim=True)
        hit = torch.zeros_like(s).scatter_(1, idx.cpu().long(), 1.0)
        size = s * (1 - s) * (own + hit * mean / total + (bal + (bal * s).sum(1, keepdim=True) / z) / z)
        assert ((d.cpu().double() - want).abs() <= size * 2.0 ** -15 + 1e-37).all()
    idx = torch.arange(k, dtype=torch.int32, device=cuda_device).repeat(T, 1).contiguous()
    for lo, hi in ((-100.0, -80.0), (-200.0, -89.0)):
        backward(lo + (hi - lo) * torch.rand((T, E), generator=g, device=cuda_device), idx)
        assert torch.isfinite(d).all()
    assert alpha or (d == 0).all()


@pytest.mark.parametrize("E,size", [(32, 4), (256, 32), (60, 12)])
def test_masks_of_the_lowest_value_beside_infinite_ones(cuda_device, E, size):
    """Sums of two of the lowest fp32 values, and differences from large keys, pass the
    fp32 range; the 64-bit keys still rank them above -inf and among themselves."""
    lowest, inf = torch.finfo(torch.float32).min, float("inf")
    n = E // size
    grp = lambda g: slice(g * size, (g + 1) * size)
    l = torch.full((8, E), -inf)
    l[0, grp(2)] = lowest                                       # one group at the lowest value, one real
    l[1, grp(1)], l[1, grp(3)] = lowest, lowest / 2             # two masked groups, by id and by key
    l[2, grp(1)], l[2, grp(3)] = lowest / 2, lowest
    l[3, 0], l[3, E - 2] = lowest, 2e38
    l[4] = lowest
    l[4, grp(3)] = lowest / 2
    l[5] = lowest
    l[5, 4], l[5, 2 * size] = 1.0, lowest / 2
    l[6] = lowest
    l[6, ::3] = -inf
    l[7] = torch.linspace(-3.4e38, -3.0e38, E)
    for t, v in ((0, 1.0), (1, 1.0), (2, 1.0), (3, 3e38), (4, 1.0)):
        l[t, E - 1] = v
        l[t, E - 2] = v / 2
    l = l.to(cuda_device)
    for topk_group, group_top in ((1, 2), (2, 2), (3, 2), (2, 1), (n, 1)):
        for k in (1, 2, 4, min(8, size)):
            idx, _, _ = run(l, None, k, (n, topk_group, group_top, 1.0), "softmax")
            want = ref.select(l.cpu(), None, k, n, topk_group, group_top, "softmax")
            assert torch.equal(idx.cpu(), want), (topk_group, group_top, k)


@pytest.mark.parametrize("E,n", [(32, 8), (250, 10), (60, 5), (256, 8)])
def test_group_scores_past_the_fp32_range(cuda_device, E, n):
    """Keys of 1e38 and more: sums of two pass the fp32 range on either side."""
    g = torch.Generator().manual_seed(51)
    up = 1e38 + 2.4e38 * torch.rand((8, E), generator=g)
    l = torch.cat([up, -up, torch.where(torch.rand((8, E), generator=g) < 0.5, up, -up)]).to(cuda_device)
    bias = 300.0 * torch.randn(E, generator=g)
    for topk_group in (1, n // 2, n - 1):
        for b in (None, bias):
            idx, _, _ = run(l, None if b is None else b.to(cuda_device), 4, (n, topk_group, 2, 1.0), "softmax")
            assert torch.equal(idx.cpu(), ref.select(l.cpu(), b, 4, n, topk_group, 2, "softmax")), topk_group
