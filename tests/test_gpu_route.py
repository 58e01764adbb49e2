"""Routing and the experts' rows against float64.

Experts, offsets, rows and slots exactly.  Weights are 64-bit values (about 1e-13 relative) rounded once to FP32; gradients
likewise, to the logits' type.  Moved rows are copies; FP32 sums of n terms are off by at most (n + 1) 2^-24 of the sum of
magnitudes, and a BF16 output rounds once more, by 2^-8."""

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from parity import say

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INF = float("inf")


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * std


def scores(x, score):
    x = x.to(F64)
    if score == "sigmoid":
        return torch.sigmoid(x)
    p = torch.softmax(x, 1)
    return torch.where(p.isnan().all(1, keepdim=True) & (x == -INF).all(1, keepdim=True), 0.0, p)


def ranks(c):
    """Position of every entry in its row, largest first, ties to the lowest index."""
    i = torch.arange(c.shape[1], device=c.device)
    ahead = (c.unsqueeze(1) > c.unsqueeze(2)) | ((c.unsqueeze(1) == c.unsqueeze(2)) & (i.view(1, 1, -1) < i.view(1, -1, 1)))
    return ahead.sum(2)


def oracle(x, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    s = scores(x, score)
    c = s + bias.to(F64) if bias is not None else (x.to(F64) if group_best == 1 or groups == 1 else s)
    T, E = c.shape
    if groups > 1:
        per = c.view(T, groups, -1)
        g = per.topk(group_best, -1).values.sum(-1)
        shut = (ranks(g) >= top_groups).repeat_interleave(E // groups, 1)
    else:
        shut = torch.zeros(T, E, dtype=torch.bool, device=x.device)
    low = torch.where(shut, torch.full_like(c, -INF), c)
    r = torch.empty(T, E, dtype=torch.long, device=x.device)
    for t in range(0, T, 256):
        r[t:t + 256] = ranks(low[t:t + 256])
    # (shut ones behind open ones that are -infinity themselves)
    r = r + shut * E
    experts = r.argsort(dim=1, stable=True)[:, :k]
    w = s.gather(1, experts)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return experts.to(torch.int32), scale * w


def close(got, want, rel):
    torch.cuda.synchronize()
    got, want = got.cpu().to(F64), want.cpu()
    assert got.shape == want.shape
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    off = (got - want).abs()
    assert bool((off <= rel * want.abs() + 1e-37)[~nan].all()), float((off / want.abs().clamp(min=1e-30))[~nan].max())


FORMS = [dict(k=1), dict(k=6), dict(k=6, renormalize=False, scale=2.5), dict(k=4, score="sigmoid"),
         dict(k=8, score="sigmoid", bias=True, scale=2.5), dict(k=3, bias=True, renormalize=False),
         dict(k=6, groups=4, top_groups=2), dict(k=8, groups=8, top_groups=4, group_best=2, bias=True, score="sigmoid"),
         dict(k=5, groups=2, top_groups=1, group_best=2), dict(k=7, groups=2, top_groups=2, score="sigmoid", renormalize=False)]


def check(x, form, seed=0):
    form = dict(form)
    E = x.shape[1]
    if form.get("bias"):
        form["bias"] = normal((E,), seed + 5, 0.1).cuda()
    want, ww = oracle(x.cuda(), **form)
    got, w = fq.route_experts(x.cuda(), **form)
    assert torch.equal(got, want)
    close(w, ww, 2.0 ** -24 + 1e-12)
    return got, w


@pytest.mark.parametrize("T,E", [(1, 8), (3, 16), (70, 64), (2100, 64), (33, 160), (2077, 160), (5, 256), (2049, 256), (40, 512),
                                 (2500, 512), (9, 72), (2060, 24)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(f"{k}{v}" for k, v in f.items()))
def test_experts_and_weights(T, E, dtype, form):
    if form["k"] > E // form.get("groups", 1) * form.get("top_groups", 1):
        pytest.skip("more choices than experts")
    say("route", T, E, dtype, form)
    check(normal((T, E), T + E, 2.0).to(dtype), form, T)  # (BF16 logits tie often)


@pytest.mark.parametrize("E,groups", [(495, 33), (510, 17), (510, 5), (504, 9), (64, 64), (128, 64), (6, 3), (7, 1), (1, 1), (511, 1)])
@pytest.mark.parametrize("T", [3, 2100])
def test_uneven_layouts(E, groups, T):
    say("route layouts", E, groups, T)
    top = (groups + 1) // 2
    check(normal((T, E), E).to(BF16), dict(k=min(6, top * (E // groups)), groups=groups, top_groups=top, score="sigmoid"))
    check(normal((T, E), E), dict(k=min(6, top * (E // groups)), groups=groups, top_groups=top, bias=True))


@pytest.mark.parametrize("T", [2, 2100])
@pytest.mark.parametrize("k", [16, 17, 64])
def test_many_choices(T, k):
    say("route many choices", T, k)
    for E in (64, 200):
        experts, w = check(normal((T, E), k), dict(k=k, score="sigmoid", renormalize=False))
        assert int(experts.sort(1).values.diff(dim=1).min()) > 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [6, 2100])
def test_switched_off_experts_and_ties(score, T):
    say("route masks", score, T)
    x = normal((T, 48), 3)
    x[0] = -INF
    x[1, 3:] = -INF                        # fewer than k left
    x[2] = 0.0                             # all equal
    x[3] = torch.finfo(F32).min            # the type's lowest value
    x[4, ::2] = -INF
    x[5] = 1e30
    x[5, 7] = 3e38
    for form in (dict(k=6), dict(k=6, renormalize=False), dict(k=6, bias=True), dict(k=6, groups=4, top_groups=2),
                 dict(k=6, groups=4, top_groups=2, group_best=2)):
        check(x, dict(form, score=score))
    experts, w = fq.route_experts(x.cuda(), 6, score=score)
    assert experts[0].tolist() == list(range(6)) and w[0].tolist() == [0.0] * 6
    assert experts[2].tolist() == list(range(6))


def test_nan_rows_stay_their_own():
    say("route nan")
    x = normal((2100, 40), 4)
    x[3, 5] = float("nan")
    x[7] = float("nan")
    x[9, 1] = INF
    for score in ("softmax", "sigmoid"):
        for form in (dict(), dict(bias=torch.zeros(40, device="cuda")), dict(groups=4, top_groups=2, group_best=2),
                     dict(renormalize=False)):
            for T in (2100, 20):
                experts, w = fq.route_experts(x[:T].cuda(), 4, score=score, **form)
                assert bool(((experts >= 0) & (experts < 40)).all())
                assert int(experts.sort(1).values.diff(dim=1).min()) > 0
                bad = w.isnan().any(1).nonzero().flatten().tolist()
                assert set(bad) <= {3, 7, 9} and 7 in bad


def test_near_scores_are_told_apart():
    """Sigmoid scores plus a bias 2^-30 apart: equal in 32 bits, not in 64."""
    say("route near scores")
    T, E = 64, 32
    x = torch.zeros(T, E)
    bias = torch.zeros(E)
    bias[5], bias[6], bias[7] = 2.0 ** -30, 2.0 ** -31, 3.0 * 2.0 ** -31
    want, _ = oracle(x.cuda(), 4, score="sigmoid", bias=bias.cuda())
    got, _ = fq.route_experts(x.cuda(), 4, score="sigmoid", bias=bias.cuda())
    assert torch.equal(got, want) and got[0].tolist() == [7, 5, 6, 0]


def test_strided_and_unaligned_logits():
    say("route strides")
    big = normal((2200, 90), 8)
    for dtype in (BF16, F32):
        for c in (0, 1, 3, 8):
            for w in (8, 64, 77):
                x = big.to(dtype).cuda()[:2101, c:c + w]
                a = fq.route_experts(x, 4, renormalize=False)
                b = fq.route_experts(x.contiguous(), 4, renormalize=False)
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
                d = normal((2101, 4), 9).cuda()
                assert torch.equal(fq.route_experts_backward(d, x, a[0], renormalize=False),
                                   fq.route_experts_backward(d, x.contiguous(), a[0], renormalize=False))


def weights_of(x, experts, score, renormalize, scale):
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    w = s.gather(1, experts.long())
    return scale * (w / w.sum(1, keepdim=True) if renormalize else w)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (77, 64, 6), (600, 256, 8), (5, 512, 64), (9, 130, 17)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient(score, renormalize, T, E, k, dtype):
    say("route gradient", score, renormalize, T, E, k, dtype)
    x, dw = normal((T, E), T, 1.5).to(dtype), normal((T, k), 2)
    experts, _ = fq.route_experts(x.cuda(), k, score=score, renormalize=renormalize)
    got = fq.route_experts_backward(dw.cuda(), x.cuda(), experts, score=score, renormalize=renormalize, scale=1.7)
    x64 = x.to(F64).requires_grad_()
    w = weights_of(x64, experts.cpu(), score, renormalize, 1.7)
    w.backward(dw.to(F64))
    want = x64.grad
    assert got.dtype == dtype
    # cancellation in d - sum d w: 1e-12 of the largest term
    scale = (1.7 * dw.abs().max()).item()
    off = (got.cpu().to(F64) - want).abs()
    step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23  # (the mean times an FP32 store; two roundings at most)
    assert bool((off <= step * want.abs() + 1e-11 * scale).all()), float(off.max())
    # the formula against differences
    if k < E and dtype == F32 and T < 100:
        g = torch.Generator().manual_seed(1)
        way = torch.randn(T, E, generator=g, dtype=F64)
        h = 1e-6
        up = (weights_of(x.to(F64) + h * way, experts.cpu(), score, renormalize, 1.7) * dw).sum()
        down = (weights_of(x.to(F64) - h * way, experts.cpu(), score, renormalize, 1.7) * dw).sum()
        slope = ((up - down) / (2 * h)).item()
        # third derivatives are below 10 a unit: h^2 10 |way|^3; rounding of the sums 1e-15 / h
        assert abs((got.cpu().to(F64) * way).sum().item() - slope) <= 1e-6 * float((want.abs() * way.abs()).sum()) + 1e-6


def test_gradient_of_rows_that_have_none():
    say("route gradient masks")
    x = normal((4, 16), 1)
    x[0] = -INF
    x[1, 2:] = -INF
    experts = torch.tensor([[0, 1, 2], [0, 1, 2], [3, -1, 4], [5, 99, 6]], dtype=torch.int32)
    dw = normal((4, 3), 2)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = fq.route_experts_backward(dw.cuda(), x.cuda(), experts.cuda(), score=score, renormalize=renorm).cpu()
            assert not d.isnan().any() and not d[0].any() and not d[1, 2:].any()
            assert bool((d[2, [3, 4]] != 0).all())


def plan(e, E):
    """Offsets, rows and slots by the definition."""
    e = e.flatten().tolist()
    slots = [i for x in range(E) for i in range(len(e)) if e[i] == x]
    rows = [-1] * len(e)
    for r, i in enumerate(slots):
        rows[i] = r
    offsets = [0]
    for x in range(E):
        offsets.append(offsets[-1] + e.count(x))
    return offsets, rows, slots + [-1] * (len(e) - len(slots))


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 64), (5, 6, 64), (63, 1, 2), (64, 2, 3), (341, 3, 512), (700, 4, 100)])
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_expert_rows(T, k, E, dropped):
    say("rows plan", T, k, E, dropped)
    g = torch.Generator().manual_seed(T)
    e = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    e[torch.rand(T, k, generator=g) < dropped] = -1
    if dropped == 0.3 and T > 5:
        e[1], e[2] = E, -(1 << 31)  # (out of range, as dropped)
    want = plan(torch.where((e < 0) | (e >= E), -1, e), E)
    got = fq.expert_rows(e.cuda(), E)
    assert got[0].dtype == torch.int64 and got[1].shape == (T, k)
    for a, b in zip(got, want):
        assert a.flatten().tolist() == b


@pytest.mark.parametrize("n,E", [(2048, 64), (2049, 64), (100003, 256), (131072, 7), (1200000, 512), (300000, 1)])
def test_expert_rows_of_many(n, E):
    say("rows plan", n, E)
    g = torch.Generator().manual_seed(n)
    e = (torch.rand(n, 1, generator=g) ** 3 * (E + 0.5)).to(torch.int32)  # (uneven; some past the last expert)
    e[torch.rand(n, 1, generator=g) < 0.01] = -7
    flat = torch.where((e < 0) | (e >= E), E, e).flatten().long()
    order = flat.sort(stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    used = int(counts.sum())
    offsets, rows, slots = (t.cpu() for t in fq.expert_rows(e.cuda(), E))
    assert torch.equal(offsets, torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))
    assert torch.equal(slots[:used].long(), order[:used]) and bool((slots[used:] == -1).all())
    back = torch.full((n,), -1, dtype=torch.int32)
    back[order[:used]] = torch.arange(used, dtype=torch.int32)
    assert torch.equal(rows.flatten(), back)


def choices(T, k, E, seed, dropped=0.2):
    g = torch.Generator().manual_seed(seed)
    e = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    e[torch.rand(T, k, generator=g) < dropped] = -1
    return e


MOVES = [(1, 1, 8), (1, 6, 2048), (5, 2, 24), (77, 3, 520), (300, 8, 2056), (33, 2, 4104), (2, 64, 16)]


@pytest.mark.parametrize("T,k,H", MOVES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gather(T, k, H, dtype):
    say("rows gather", T, k, H, dtype)
    e = choices(T, k, 64, T)
    _, rows, slots = fq.expert_rows(e.cuda(), 64)
    x = normal((T, H + 8), T).to(dtype).cuda()[:, :H]
    out = torch.full((T * k + 1, H + 8), 3.0, dtype=dtype, device="cuda")
    fq.fp8bq_gather_rows(x, slots, k, out[:T * k, :H])
    s = slots.long()
    want = torch.where((s >= 0).unsqueeze(1), x[s.clamp(min=0) // k], 0)
    assert torch.equal(out[:T * k, :H], want) and torch.equal(fq.gather_rows(x.contiguous(), slots, k), want)
    assert bool((out[T * k] == 3.0).all() and (out[:, H:] == 3.0).all())


@pytest.mark.parametrize("T,k,H", MOVES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, H, dtype, out, weighted):
    say("rows combine", T, k, H, dtype, out, weighted)
    _, rows, slots = fq.expert_rows(choices(T, k, 64, T).cuda(), 64)
    y = normal((T * k, H), 1).to(dtype).cuda()
    y[slots.long() < 0] = float("nan")  # (rows of no choice are not read)
    w = normal((T, k), 2).cuda() if weighted else None
    r = rows.long()
    each = torch.where((r >= 0).unsqueeze(2), y[r.clamp(min=0)].to(F64), 0.0)
    each = each * (w.to(F64).unsqueeze(2) if weighted else 1.0)
    got = fq.combine_rows(y, rows, w, out_dtype=out)
    want = each.sum(1)
    torch.cuda.synchronize()
    limit = (k + 1) * 2.0 ** -24 * each.abs().sum(1) + (2.0 ** -8 * want.abs() if out == BF16 else 0.0)
    assert got.dtype == out and bool(((got.to(F64) - want).abs() <= 1.01 * limit).all())


@pytest.mark.parametrize("T,k,H", MOVES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dout_type", [BF16, F32])
def test_combine_backward(T, k, H, dtype, dout_type):
    say("rows combine backward", T, k, H, dtype, dout_type)
    _, rows, slots = fq.expert_rows(choices(T, k, 64, T).cuda(), 64)
    y = normal((T * k, H), 1).to(dtype).cuda()
    y[slots.long() < 0] = float("nan")
    w, d = normal((T, k), 2).cuda(), normal((T, H), 3).to(dout_type).cuda()
    dy, dw = fq.combine_rows_backward(d, y, rows, w, slots)
    s, r = slots.long(), rows.long()
    want = torch.where((s >= 0).unsqueeze(1), d[s.clamp(min=0) // k].to(F64) * w.flatten()[s.clamp(min=0)].to(F64).unsqueeze(1), 0.0)
    assert dy.dtype == dtype
    assert bool(((dy.to(F64) - want).abs() <= (2.0 ** -8 + 2.0 ** -24 if dtype == BF16 else 2.0 ** -24) * want.abs()).all())
    terms = torch.where((r >= 0).unsqueeze(2), y[r.clamp(min=0)].to(F64), 0.0) * d.to(F64).unsqueeze(1)
    assert bool(((dw.to(F64) - terms.sum(2)).abs() <= (H + 1) * 2.0 ** -24 * terms.abs().sum(2)).all())


def test_layer_forward_and_gradients():
    """Router, rows, experts and their sum as a training step chains them, against autograd in 64 bits (experts that scale
    their rows, so that only what is tested here rounds)."""
    say("route layer")
    T, E, k, H = 200, 16, 3, 64
    x, router, gain = normal((T, H), 1).cuda(), normal((H, E), 2, 0.2).cuda(), normal((E,), 3).cuda()
    dout = normal((T, H), 4).cuda()
    logits = x @ router
    experts, w = fq.route_experts(logits, k, score="sigmoid", scale=1.5)
    offsets, rows, slots = fq.expert_rows(experts, E)
    xs = fq.gather_rows(x, slots, k)
    of_row = gain.repeat_interleave(offsets.diff()).unsqueeze(1)
    y = xs * of_row
    out = fq.combine_rows(y, rows, w)
    dy, dw = fq.combine_rows_backward(dout, y, rows, w, slots)
    dx = fq.combine_rows(dy * of_row, rows)
    dlogits = fq.route_experts_backward(dw, logits, experts, score="sigmoid", scale=1.5)

    x64, l64 = x.to(F64).requires_grad_(), logits.to(F64).requires_grad_()
    w64 = weights_of(l64, experts, "sigmoid", True, 1.5)
    o64 = sum(w64[:, j:j + 1] * gain.to(F64)[experts[:, j].long()].unsqueeze(1) * x64 for j in range(k))
    o64.backward(dout.to(F64))
    torch.cuda.synchronize()
    # sums of H = 64 products of rounded factors, whose magnitudes add up to at most 16 of the largest result
    for got, want in ((out, o64.detach()), (dx, x64.grad), (dlogits, l64.grad)):
        assert float((got.to(F64) - want).abs().max()) <= (H + 4) * 2.0 ** -24 * 16 * float(want.abs().max())


@pytest.mark.parametrize("T", [3, 3000])
def test_captured_and_replayed(T):
    say("route graph", T)
    E, k, H = 64, 4, 256

    def step(x, y, dout):
        experts, w = fq.route_experts(x, k, score="sigmoid", groups=4, top_groups=2, group_best=2)
        offsets, rows, slots = fq.expert_rows(experts, E)
        dy, dw = fq.combine_rows_backward(dout, y, rows, w, slots)
        return (experts, w, offsets, rows, slots, fq.gather_rows(dout, slots, k), fq.combine_rows(y, rows, w), dy, dw,
                fq.route_experts_backward(dw, x, experts, score="sigmoid"))

    x, y, d = normal((T, E), 1).cuda(), normal((T * k, H), 2).to(BF16).cuda(), normal((T, H), 3).to(BF16).cuda()
    step(x, y, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(x, y, d)
    for seed in range(3):
        x.copy_(normal((T, E), 10 + seed))
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        for a, b in zip(got, step(x, y, d)):
            assert torch.equal(a, b)


def test_no_tokens():
    say("route empty")
    z = torch.zeros
    experts, w = fq.route_experts(z((0, 8), device="cuda"), 2)
    assert experts.shape == w.shape == (0, 2)
    offsets, rows, slots = fq.expert_rows(experts, 8)
    assert offsets.tolist() == [0] * 9 and rows.shape == (0, 2) and slots.shape == (0,)
    x = z((0, 16), device="cuda")
    assert fq.gather_rows(x, slots, 2).shape == (0, 16) and fq.combine_rows(x, rows, w).shape == (0, 16)
