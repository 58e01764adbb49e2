"""Measured cases of expert routing, the experts' rows, the 8-bit linear layer and the orthogonalized update.

Four operators, on the sizes of a 2B-class decoder (hidden 2048, QKV 2560, SwiGLU 2 x 5632) and of experts cut from
its feed-forward layer (1408 = 5632 / 4 wide):

  route   experts and weights of each token from the router's logits [T, E]; in training also the logits' gradient.
          s = softmax or sigmoid of the logits, c = s + bias; a group of E / G experts scores the sum of its best one
          or two c, the best `top_groups` groups stay, and of their experts the k with the largest c are taken,
          descending, ties to the lowest index.  w = scale s, or scale s / sum of the chosen s (zero where that sum is).
  rows    the way of the tokens' rows to the experts and back: a stable sort of the T k choices by expert (choices of -1
          go nowhere), the sorted rows, the weighted sum of the experts' rows, and in training both gradients.
  int8    y = sa sb Q(x) . Qw^T in 8-bit integers, one scale for each token and each output channel: s = max(amax / 127,
          1e-12), codes fp32(x / s) to the nearest, ties to even; dense, grouped by expert, and a step's gradients
          dx = Q(dy) . Q(W^T)^T and dw = Q(dy^T) . Q(x^T)^T.
  ortho   Newton-Schulz orthogonalization of each matrix of a batch: X = G / (|G| + eps), then five times
          X = a X + (b A + c A^2) X with A = X X^T (on the shorter side), a, b, c = 3.4445, -4.7750, 2.0315.
"""

import torch

own = False

BF16 = torch.bfloat16
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS, EPS = 5, 1e-7


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one token on 64 experts, six of them: the decode step of one sequence
        dict(name="route_1", op="route", T=1, E=64, k=6, score="softmax", bias=False, G=1, top=1, best=1, renorm=True,
             masked=0, x="f32", train=False),
        # training micro-batch, balanced by a bias, experts in eight groups of which a token uses four
        dict(name="route_groups_16384", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, G=8, top=4, best=2,
             renorm=True, masked=0, x="f32", train=True),
        # odd batch with BF16 logits, eleven experts switched off, weights as the softmax gives them
        dict(name="route_8191", op="route", T=8191, E=96, k=2, score="softmax", bias=False, G=1, top=1, best=1,
             renorm=False, masked=11, x="bf16", train=True),
        # five decoding sequences, six experts of 64 each
        dict(name="rows_5", op="rows", T=5, k=6, E=64, H=2048, dropped=0.0, train=False),
        # training micro-batch, two experts a token; some choices dropped (an expert over its capacity, padding)
        dict(name="rows_16384", op="rows", T=16384, k=2, E=64, H=2048, dropped=0.03, train=True),
        # one token through gate+up: the decode step of one sequence
        dict(name="int8_1", op="int8", M=1, N=11264, K=2048, x="bf16"),
        # a prompt batch through gate+up: the largest product
        dict(name="int8_16384", op="int8", M=16384, N=11264, K=2048, x="bf16"),
        # gradients of the down projection; the tokens end inside every kind of tile
        dict(name="int8_backward_4099", op="int8_backward", M=4099, N=2048, K=5632, x="bf16"),
        # 128 decoding sequences, six experts of 64 each
        dict(name="int8_experts_768", op="int8_experts", E=64, T=768, N=2816, K=2048, skew=0.4, x="bf16"),
        # a small expert layer's eight stacked down projections
        dict(name="ortho_8x512x384", op="ortho", B=8, R=512, C=384, rank=32, x="bf16"),
        # the gate+up weight of one layer, FP32 momentum
        dict(name="ortho_11264x2048", op="ortho", B=1, R=11264, C=2048, rank=256, x="f32"),
        # stacked experts of one layer, wide matrices
        dict(name="ortho_32x1408x2048", op="ortho", B=32, R=1408, C=2048, rank=64, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("route", "route", "rows", "rows", "int8", "int8_backward", "int8_experts", "ortho", "ortho"))
    x = rng.choice(("bf16", "bf16", "f32"))
    if op == "route":
        G = rng.choice((1, 1, 2, 4, 6, 8))
        per = _log(rng, 8 if G == 1 else 2, 256 // G)
        best = 1 if per < 2 else rng.choice((1, 2))
        top = G if G == 1 else rng.randint(1, G)
        bias = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 16384), E=G * per, k=rng.randint(1, min(8, top * per)),
                    score=rng.choice(("softmax", "sigmoid")), bias=bias, G=G, top=top, best=best,
                    renorm=rng.random() < 0.7, masked=rng.choice((0, 0, G * per // 8)), x=x, train=rng.random() < 0.5)
    if op == "rows":
        k = rng.randint(1, 8)
        return dict(op=op, T=_log(rng, 1, 16384 * 2 // k), k=k, E=max(k, _log(rng, 2, 256)), H=8 * _log(rng, 16, 256),
                    dropped=rng.choice((0.0, 0.03, 0.5)), train=rng.random() < 0.5)
    if op == "int8":
        return dict(op=op, M=_log(rng, 1, 8192), N=8 * _log(rng, 32, 1408), K=16 * _log(rng, 16, 352), x=x)
    if op == "int8_backward":
        return dict(op=op, M=_log(rng, 64, 4099), N=16 * _log(rng, 16, 128), K=16 * _log(rng, 16, 352), x=x)
    if op == "int8_experts":
        return dict(op=op, E=_log(rng, 4, 64), T=_log(rng, 1, 4096), N=8 * _log(rng, 32, 352), K=16 * _log(rng, 16, 128),
                    skew=rng.choice((0.0, 0.4, 1.0)), x=x)
    while True:
        R, C = _log(rng, 64, 11264), _log(rng, 64, 2816)
        c = dict(op=op, B=_log(rng, 1, 16), R=R, C=C, rank=_log(rng, 1, max(2, min(R, C) // 4)), x=x)
        if c["B"] * R * C <= 11264 * 2048 and work(c)["flops"] <= 1.1e12:
            return c


def _counts(case):
    """Tokens per expert, most first: shares proportional to rank^-skew, largest remainders rounded up."""
    E, T = case["E"], case["T"]
    share = [(e + 1.0) ** -case["skew"] for e in range(E)]
    total = sum(share)
    exact_ = [T * s / total for s in share]
    n = [int(v) for v in exact_]
    left = sorted(range(E), key=lambda e: (n[e] - exact_[e], e))[:T - sum(n)]
    return [n[e] + (e in left) for e in range(E)]


def work(case):
    op = case["op"]
    xb = 2 if case.get("x") != "f32" else 4
    if op == "route":  # logits in; experts and weights out; the weights' gradient in, the logits' out
        T, E, k = case["T"], case["E"], case["k"]
        n = T * E * xb + 8 * T * k
        return dict(bytes=n + (T * E * xb + 4 * T * k if case["train"] else 0), flops=10.0 * T * E)
    if op == "rows":  # x in, rows out, rows in, sum out; backward: its gradient and the rows in, three gradients out
        T, k, H = case["T"], case["k"], case["H"]
        held = T * k * (1.0 - case["dropped"])
        n = 2 * H * (T + T * k + held + T) + 16 * T * k
        if case["train"]:
            n += 2 * H * (T + held + T * k) + 2 * H * (held + T) + 4 * T * k
        return dict(bytes=n, flops=2.0 * held * H * (3 if case["train"] else 1))
    if op == "ortho":
        B, m, n = case["B"], min(case["R"], case["C"]), max(case["R"], case["C"])
        return dict(bytes=B * m * n * (xb + 2), flops=B * STEPS * (4.0 * m * m * n + 2.0 * m ** 3))
    N, K = case["N"], case["K"]
    if op == "int8":
        M = case["M"]
        return dict(bytes=M * K * xb + N * (K + 4) + 2 * M * N, flops=2.0 * M * N * K)
    if op == "int8_backward":  # dy, x and W^T in; dx and dw out
        M = case["M"]
        return dict(bytes=(M * N + M * K) * xb + K * (N + 4) + 2 * M * K + 2 * N * K, flops=4.0 * M * N * K)
    T = case["T"]
    used = sum(n > 0 for n in _counts(case))
    return dict(bytes=T * K * xb + used * N * (K + 4) + 2 * T * N, flops=2.0 * T * N * K)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _normal(g, shape, std, outliers=False):
    t = torch.randn(shape, generator=g, device="cuda") * std
    if outliers:  # a hundredth of the channels fifty times larger
        t[:, torch.randperm(shape[1], generator=g, device="cuda")[:shape[1] // 100]] *= 50.0
    return t


def _on(t, v):
    """v as a tensor on t's device: a division by a Python number is a product with its rounded reciprocal there."""
    return torch.full((), v, dtype=torch.float32, device=t.device)


def _to_int8(w):
    """Codes [R, C] and scales [R] of w, one scale a row."""
    s = (w.float().abs().amax(1) / _on(w, 127.0)).clamp(min=1e-12)
    return torch.round(w.float() / s.unsqueeze(1)).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    kind = BF16 if case.get("x") == "bf16" else torch.float32
    if op == "route":
        T, E = case["T"], case["E"]
        x = _normal(g, (T, E), 1.5) + _normal(g, (1, E), 0.5)  # some experts are liked by most tokens
        if case["masked"]:
            x[:, torch.randperm(E, generator=g, device="cuda")[:case["masked"]]] = float("-inf")
        s["logits"] = x.to(kind)
        s["b"] = _normal(g, (E,), 0.05) if case["bias"] else None
        s["dw"] = _normal(g, (T, case["k"]), 1e-2)
        s["factor"] = 2.5
    elif op == "rows":
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        like = _normal(g, (T, E), 1.0) + _normal(g, (1, E), 0.5)
        e = like.topk(k, 1).indices.to(torch.int32)
        e[torch.rand(T, k, generator=g, device="cuda") < case["dropped"]] = -1
        s["experts"] = e.contiguous()
        w = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["x"] = _normal(g, (T, H), 1.0).to(BF16)
        s["y"] = _normal(g, (T * k, H), 1.0).to(BF16)  # what the experts answer
        s["dout"] = _normal(g, (T, H), 1e-3).to(BF16)
        s["dgathered"] = _normal(g, (T * k, H), 1e-3).to(BF16)
    elif op == "ortho":
        B, R, C, r = case["B"], case["R"], case["C"], case["rank"]
        # a gradient: mostly of low rank, its leading directions much stronger, and noise of all the tokens
        u = torch.randn(B, R, r, generator=g, device="cuda") / torch.arange(1, r + 1, device="cuda").sqrt()
        v = torch.randn(B, r, C, generator=g, device="cuda")
        s["g"] = ((torch.bmm(u, v) + 0.2 * torch.randn(B, R, C, generator=g, device="cuda")) * 1e-4).to(kind)
    else:
        N, K = case["N"], case["K"]
        if op == "int8_experts":
            n = torch.tensor(_counts(case), device="cuda")[torch.randperm(case["E"], generator=g, device="cuda")]
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)])
        M, E = (case["T"], case["E"]) if op == "int8_experts" else (case["M"], 1)
        s["x"] = _normal(g, (M, K), 1.0, True).to(kind)
        w = _normal(g, (E * N, K), 0.02).to(BF16)
        if op == "int8_backward":
            s["dy"] = _normal(g, (M, N), 1e-3).to(kind)
            s["qwt"], s["swt"] = _to_int8(w.t().contiguous())
        else:
            s["qw"], s["sw"] = _to_int8(w)
    return s


# ---------------------------------------------------------------------------------------------
# the plain form: elementary operations in 32 bits; the choice of experts in 64, where near values are told apart
# ---------------------------------------------------------------------------------------------

def _plain_route(s):
    x = s["logits"].double()
    T, E = x.shape
    G, k = s["G"], s["k"]
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    c = p if s["b"] is None else p + s["b"].double()
    if G > 1:
        score = c.view(T, G, E // G).sort(-1, descending=True).values[..., :s["best"]].sum(-1)
        kept = score.sort(dim=-1, descending=True, stable=True).indices[:, :s["top"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        c = torch.where(open_.repeat_interleave(E // G, 1), c, -torch.inf)
    experts = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    p = p.float()
    chosen = p.gather(1, experts)
    total = chosen.sum(1, keepdim=True)
    if s["renorm"]:
        chosen = torch.where(total > 0, chosen / total, 0.0)
    weights = s["factor"] * chosen
    if not s["train"]:
        return experts.to(torch.int32), weights
    d = s["factor"] * s["dw"]
    if s["renorm"]:
        d = torch.where(total > 0, (d - (d * chosen).sum(1, keepdim=True)) / total, 0.0)
    dp = torch.zeros_like(p).scatter_(1, experts, d)
    if s["score"] == "softmax":
        dx = p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        dx = dp * p * (1.0 - p)
    return experts.to(torch.int32), weights, dx.to(s["logits"].dtype)


def _plain_rows(s):
    e, k, E = s["experts"].flatten().long(), s["k"], s["E"]
    T, H = s["x"].shape
    n = e.numel()
    order = torch.where(e < 0, E, e).sort(stable=True).indices
    counts = torch.bincount(torch.where(e < 0, E, e), minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(n, device=e.device)
    in_use = place < offsets[E]
    slots = torch.where(in_use, order, -1)
    rows = torch.empty_like(order).index_copy_(0, order, place)
    rows = torch.where(e < 0, -1, rows)
    held = (rows >= 0).unsqueeze(1)
    gathered = torch.where(in_use.unsqueeze(1), s["x"][order // k], 0)

    def combined(y, w):
        each = torch.where(held, y[rows.clamp(min=0)].float(), 0.0)
        return ((each * w.reshape(-1, 1)) if w is not None else each).view(T, k, H).sum(1).to(BF16)

    out = combined(s["y"], s["weights"])
    result = (offsets, rows.view(T, k).to(torch.int32), slots.to(torch.int32), gathered, out)
    if not s["train"]:
        return result
    d = s["dout"].float()
    dy = torch.where(in_use.unsqueeze(1), d[order // k] * s["weights"].flatten()[order].unsqueeze(1), 0.0).to(BF16)
    dw = torch.where(held, s["y"][rows.clamp(min=0)].float(), 0.0).view(T, k, H)
    dw = (dw * d.unsqueeze(1)).sum(-1)
    return result + (dy, dw, combined(s["dgathered"], None))


def _rounded(x):
    """What the 8-bit codes of x stand for without their scale, and the scale, one a row."""
    v = x.float()
    s = (v.abs().amax(1, keepdim=True) / _on(v, 127.0)).clamp(min=1e-12)
    return torch.round(v / s), s


def _plain_int8(s):
    op, N = s["op"], s["N"]
    if op == "int8":
        q, sx = _rounded(s["x"])
        return ((q @ s["qw"].float().t()) * sx * s["sw"]).to(BF16)
    if op == "int8_backward":
        q, sd = _rounded(s["dy"])
        dx = (q @ s["qwt"].float().t()) * sd * s["swt"]
        qd, sd = _rounded(s["dy"].t())
        qx, sx = _rounded(s["x"].t())
        return dx.to(BF16), ((qd @ qx.t()) * sd * sx.t()).to(BF16)
    # tokens laid out as [experts in use, most tokens of one, width], zeros where an expert has fewer
    E, off, K = s["E"], s["offsets"], s["K"]
    n = off[1:] - off[:-1]
    used = n.nonzero().squeeze(1)
    place = torch.arange(int(n.max()), device=off.device)
    rows = off[used].unsqueeze(1) + place
    held = place < n[used].unsqueeze(1)
    q, sx = _rounded(s["x"])
    q = torch.where(held.unsqueeze(-1), q[torch.where(held, rows, 0)], 0.0)
    w = s["qw"].view(E, N, K)[used].float()
    y = torch.bmm(q, w.transpose(1, 2).contiguous()) * s["sw"].view(E, 1, N)[used]
    return (y[held] * sx).to(BF16)


def _plain_ortho(s):
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        A = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    return (x.transpose(1, 2).contiguous() if tall else x).to(BF16)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["op"]
    if not own:
        return (_plain_route if op == "route" else _plain_rows if op == "rows" else
                _plain_ortho if op == "ortho" else _plain_int8)(s)
    import fp8_blockwise_quantized_amd as fq
    if op == "route":
        how = dict(score=s["score"], renormalize=s["renorm"], scale=s["factor"])
        experts, weights = fq.route_experts(s["logits"], s["k"], bias=s["b"], groups=s["G"], top_groups=s["top"],
                                            group_best=s["best"], **how)
        if not s["train"]:
            return experts, weights
        return experts, weights, fq.route_experts_backward(s["dw"], s["logits"], experts, **how)
    if op == "rows":
        offsets, rows, slots = fq.expert_rows(s["experts"], s["E"])
        result = (offsets, rows, slots, fq.gather_rows(s["x"], slots, s["k"]), fq.combine_rows(s["y"], rows, s["weights"]))
        if not s["train"]:
            return result
        return result + fq.combine_rows_backward(s["dout"], s["y"], rows, s["weights"], slots) + (
            fq.combine_rows(s["dgathered"], rows),)
    if op == "ortho":
        return fq.orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    if op == "int8":
        return fq.linear_int8(s["x"], s["qw"], s["sw"])
    if op == "int8_experts":
        return fq.grouped_linear_int8(s["x"], s["offsets"], s["qw"], s["sw"])
    dx = fq.gemm_int8(*fq.quantize_int8(s["dy"]), s["qwt"], s["swt"])
    return dx, fq.gemm_int8(*fq.quantize_int8_t(s["dy"]), *fq.quantize_int8_t(s["x"]))


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_route(s):
    x = s["logits"].double()
    T, E = x.shape
    G, k, f = s["G"], s["k"], s["factor"]
    p = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
    c = p if s["b"] is None else p + s["b"].double()
    index = torch.arange(E, device=x.device)
    closed = torch.zeros(T, E, dtype=torch.bool, device=x.device)
    if G > 1:
        per = c.view(T, G, -1)
        score = per.max(-1).values
        if s["best"] == 2:
            first = per.argmax(-1, keepdim=True)
            score = score + per.scatter(-1, first, -torch.inf).max(-1).values
        group = torch.arange(G, device=x.device)
        ahead = (score.unsqueeze(1) > score.unsqueeze(2)) | (
            (score.unsqueeze(1) == score.unsqueeze(2)) & (group.view(1, 1, G) < group.view(1, G, 1)))
        closed = (ahead.sum(2) >= s["top"]).repeat_interleave(E // G, 1)
    experts = torch.empty(T, k, dtype=torch.long, device=x.device)
    left = torch.where(closed, -torch.inf, c)
    taken = closed.clone()
    for j in range(k):
        top = torch.where(taken, -torch.inf, left).max(1, keepdim=True).values
        first = torch.where((left >= top) & ~taken, index, E).min(1).values
        experts[:, j] = first
        taken.scatter_(1, first.unsqueeze(1), True)
    w = p.gather(1, experts)
    total = w.sum(1, keepdim=True)
    live = total > 0
    if s["renorm"]:
        w = torch.where(live, w / total, 0.0)
    if not s["train"]:
        return experts.to(torch.int32), f * w
    d = f * s["dw"].double()
    if s["renorm"]:
        d = torch.where(live, (d - (d * w).sum(1, keepdim=True)) / total, 0.0)
    dp = torch.zeros_like(p).scatter(1, experts, d)
    dx = p * (dp - (p * dp).sum(1, keepdim=True)) if s["score"] == "softmax" else dp * p * (1 - p)
    return experts.to(torch.int32), f * w, dx


def _exact_rows(s):
    e = s["experts"].cpu()
    T, k, E = e.shape[0], s["k"], s["E"]
    slots = torch.full((T * k,), -1, dtype=torch.int32)
    rows = torch.full((T * k,), -1, dtype=torch.int32)
    offsets, at = [0], 0
    for x in range(E):
        mine = (e.flatten() == x).nonzero().squeeze(1)
        slots[at:at + len(mine)] = mine.to(torch.int32)
        rows[mine] = torch.arange(at, at + len(mine), dtype=torch.int32)
        at += len(mine)
        offsets.append(at)
    dev = s["x"].device
    slots, rows, used = slots.to(dev), rows.to(dev).view(T, k), slots[:at].to(dev).long()
    gathered = torch.zeros(T * k, s["H"], dtype=torch.float64, device=dev)
    gathered[:at] = s["x"][used // k].double()
    w, d = s["weights"].double(), s["dout"].double()

    def combined(y, w):
        out = torch.zeros(T, s["H"], dtype=torch.float64, device=dev)
        for j in range(k):
            has = rows[:, j] >= 0
            out[has] += w[has, j].unsqueeze(1) * y[rows[has, j].long()].double()
        return out

    result = (torch.tensor(offsets, device=dev), rows, slots, gathered, combined(s["y"], w))
    if not s["train"]:
        return result
    dy = torch.zeros(T * k, s["H"], dtype=torch.float64, device=dev)
    dy[:at] = d[used // k] * w.flatten()[used].unsqueeze(1)
    dw = torch.zeros(T, k, dtype=torch.float64, device=dev)
    for j in range(k):
        has = rows[:, j] >= 0
        dw[has, j] = (d[has] * s["y"][rows[has, j].long()].double()).sum(1)
    return result + (dy, dw, combined(s["dgathered"], torch.ones_like(w)))


def _exact_codes(x):
    """Codes and scales of x's rows; the scale and the quotient are 32-bit values."""
    v = x.double()
    s = torch.maximum((v.abs().max(1, keepdim=True).values / 127.0).float(), torch.tensor(1e-12, device=x.device)).double()
    y = (v / s).float().double()
    low = torch.floor(y)
    up = (y - low > 0.5) | ((y - low == 0.5) & (low % 2 != 0))
    return low + up, s


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "route":
        return _exact_route(s)
    if op == "rows":
        return _exact_rows(s)
    if op == "ortho":
        out = []
        for g in s["g"].double():
            x = g / (torch.linalg.matrix_norm(g) + EPS)
            a, b, c = COEFFICIENTS
            for _ in range(STEPS):
                if x.shape[0] > x.shape[1]:
                    A = x.t() @ x
                    x = a * x + b * (x @ A) + c * (x @ (A @ A))
                else:
                    A = x @ x.t()
                    x = a * x + b * (A @ x) + c * ((A @ A) @ x)
            out.append(x)
        return torch.stack(out)
    if op == "int8_backward":
        q, sd = _exact_codes(s["dy"])
        dx = q @ s["qwt"].double().t() * sd * s["swt"].double()
        (qd, sd), (qx, sx) = _exact_codes(s["dy"].t()), _exact_codes(s["x"].t())
        return dx, qd @ qx.t() * sd * sx.t()
    q, sx = _exact_codes(s["x"])
    if op == "int8":
        return q @ s["qw"].double().t() * sx * s["sw"].double()
    off, N = s["offsets"].tolist(), s["N"]
    y = torch.zeros(s["T"], N, dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        a, b = off[e], off[e + 1]
        if b > a:
            y[a:b] = q[a:b] @ s["qw"][e * N:(e + 1) * N].double().t() * sx[a:b] * s["sw"][e * N:(e + 1) * N].double()
    return y
