"""Cases for timing and checking the block's routing and 4-bit operators.

Four operators:

* select: routing to experts from the router's logits (softmax or sigmoid
  scores, selection bias, groups, top-k, renormalised weights);
* select_backward: its gradient with respect to all logits, with that of the
  balance loss;
* balance_loss: the loss that evens out the experts' load;
* experts: the SwiGLU experts' products with 4-bit weights (E2M1 codes, one
  E8M0 scale per 32 weights along k).

``run`` computes a case in plain torch operations, or, where ``own`` is true,
with the library's calls; ``exact`` computes the same from the definitions in
64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32          # weights per scale
BLOCK_EXPERTS = 256  # experts of the block
COEF = 1e-2         # factor of the balance loss
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# E2M1 magnitudes by code; codes 8-15 are their negatives
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
def listed():
    route = dict(experts=256, topk=8, dtype="fp32", score="softmax", renormalize=True, masked=0.0,
                 padded=0.0)
    select = dict(route, op="select", groups=1, topk_groups=1, group_best=2, bias=False)
    grad = dict(route, op="select_backward", balance=True)
    loss = dict(route, op="balance_loss")
    experts = dict(op="experts", hidden=5120, inter=2560, topk=8, skew=False)
    return [
        # a decode batch of the block's own routing rule, balanced by a bias: latency
        dict(select, name="select_decode", tokens=32, score="sigmoid", groups=8, topk_groups=4,
             bias=True),
        # a long prefill of a softmax router
        dict(select, name="select_prefill", tokens=16384),
        # bf16 logits (many ties), experts that are switched off, odd counts, raw weights
        dict(select, name="select_odd", tokens=1537, experts=60, topk=5, groups=3, topk_groups=2,
             group_best=1, dtype="bf16", masked=0.1, renormalize=False),
        # the gradient at a training micro-batch, balance loss included
        dict(grad, name="select_grad_micro", tokens=4096),
        # raw sigmoid weights of few experts, padded rows, bf16 logits
        dict(grad, name="select_grad_odd", tokens=509, experts=60, topk=4, dtype="bf16",
             score="sigmoid", renormalize=False, balance=False, padded=0.2),
        # the loss at a training micro-batch, and on a padded batch of few experts
        dict(loss, name="balance_micro", tokens=4096),
        dict(loss, name="balance_odd", tokens=333, experts=160, topk=6, dtype="bf16",
             score="sigmoid", padded=0.2),
        # one sequence's next token
        dict(experts, name="experts_one", tokens=1),
        # a decode batch
        dict(experts, name="experts_decode", tokens=32),
        # many sequences, or a short prompt
        dict(experts, name="experts_mid", tokens=512),
        # a prefill chunk: the largest
        dict(experts, name="experts_prefill", tokens=4096),
        # a small model, uneven load, a last row block of odd length
        dict(experts, name="experts_small", tokens=203, hidden=768, inter=384, topk=5, skew=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select_backward", "balance_loss", "experts", "experts"])
    if op == "experts":
        hidden, inter = 256 * rng.randint(1, 20), 128 * rng.randint(1, 20)
        return dict(op=op, tokens=_log(rng, 1, 4096), hidden=hidden, inter=inter,
                    topk=rng.randint(1, 8), skew=rng.random() < 0.4)
    experts = rng.choice([256, 256, 64, 128, 512, rng.randint(2, 40), rng.randint(2, 512)])
    case = dict(op=op, tokens=_log(rng, 1, min(16384, 16384 * 256 // experts)), experts=experts,
                topk=rng.randint(1, min(8, experts)), dtype=rng.choice(["fp32", "bf16"]),
                score=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.6,
                masked=rng.choice([0.0, 0.0, 0.1]), padded=rng.choice([0.0, 0.0, 0.2]))
    if op == "select":
        groups = rng.choice([g for g in range(1, min(64, experts) + 1) if experts % g == 0])
        least = -(-case["topk"] // (experts // groups))
        case.update(padded=0.0, groups=groups, topk_groups=rng.randint(least, groups),
                    group_best=rng.randint(1, 2), bias=rng.random() < 0.5)
    if op == "select_backward":
        case["balance"] = rng.random() < 0.5
    return case


def _touched(case):
    """Experts that a batch is expected to reach (_ids draws without putting back)."""
    hot, heavy = (16.0, math.exp(4.0)) if case["skew"] else (0.0, 1.0)
    cold = BLOCK_EXPERTS - hot
    total = {"hot": hot, "cold": cold}
    for _ in range(case["topk"]):
        p = hot * heavy / (hot * heavy + cold)
        hot, cold = max(0.0, hot - p), cold - (1 - p)
    left = {"hot": hot, "cold": cold}
    return sum(n * (1 - (left[k] / n) ** case["tokens"]) for k, n in total.items() if n)


def work(case):
    T, k = case["tokens"], case["topk"]
    if case["op"] == "experts":
        H, I = case["hidden"], case["inter"]
        return {"bytes": _touched(case) * 3 * H * I * (0.5 + 1 / GROUP) + 2 * T * H + 2 * T * k * H
                + 4 * T * k, "flops": 6 * T * k * H * I}
    E, size = case["experts"], 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "select":
        return {"bytes": T * E * size + 8 * T * k + (4 * E if case["bias"] else 0),
                "flops": 4 * T * E}
    if case["op"] == "select_backward":
        return {"bytes": 2 * T * E * size + 8 * T * k + (4 * E if case["balance"] else 0),
                "flops": 8 * T * E}
    return {"bytes": T * E * size + 4 * T * k + 4 * E, "flops": 4 * T * E}


# ---------------------------------------------------------------------------
# inputs
def _ids(T, E, k, g, skew=False, padded=0.0):
    """Expert ids [T, k]: k different experts per token, -1 throughout a padded row."""
    score = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp_(1e-9, 1 - 1e-6)))
    if skew:  # sixteen experts take most of the tokens
        score[:, 5::16] += 4.0
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    if padded:
        ids[torch.rand(T, generator=g, device=DEV) < padded] = -1
    return ids


def _quantize(w):
    """Codes [N, K / 2] (two a byte, the lower k in the low half) and E8M0 scales
    [N, K / 32] of w [N, K]: the least power of two (2^-126 or more) by which the
    group's largest magnitude is at most 7, codes to the nearest, ties to even."""
    n, k = w.shape
    groups = w.view(n, k // GROUP, GROUP)
    mantissa, exponent = torch.frexp(groups.abs().amax(2))
    scale = torch.where(mantissa > 0, exponent + 124 + (mantissa > 0.875).int(), 1).clamp_(min=1)
    y = (groups * torch.exp2((127 - scale).float())[:, :, None]).view(n, k)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)) | ((y < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)

    st, T, k = dict(case), case["tokens"], case["topk"]
    if case["op"] == "experts":
        return _prepare_experts(st, normal, _ids(T, BLOCK_EXPERTS, k, g, case["skew"]))
    E = case["experts"]
    z = normal(T, E, scale=1.5)
    z += normal(E, scale=0.5)  # some experts are liked more
    if case["masked"]:
        z[torch.rand(T, E, generator=g, device=DEV) < case["masked"]] = -math.inf
    st["logits"] = z.to(_TYPES[case["dtype"]])
    if case["op"] == "select":
        # as large as the scores' own spread
        spread = 0.3 if case["score"] == "sigmoid" else 2.0 / E
        st["sel_bias"] = normal(E, scale=spread) if case["bias"] else None
        return st
    st["ids"] = _ids(T, E, k, g, padded=case["padded"])
    if case["op"] == "select_backward":
        st["grad"] = normal(T, k, scale=1e-2)
        st["load"] = st["grad_loss"] = None
        if case["balance"]:
            st["load"] = COEF * (0.2 + torch.rand(E, generator=g, device=DEV)) / T
            st["grad_loss"] = torch.full((), 0.5, device=DEV)  # of several micro-batches
    return st


def _prepare_experts(st, normal, ids):
    T, k, H, I = st["tokens"], st["topk"], st["hidden"], st["inter"]
    E = BLOCK_EXPERTS
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    st.update(x=normal(T, H, dtype=torch.bfloat16), offsets=offsets, bounds=offsets.tolist(),
              src=torch.argsort(flat, stable=True).to(torch.int32))
    empty = dict(dtype=torch.uint8, device=DEV)
    q = {"gate_up": (torch.empty(E, 2 * I, H // 2, **empty),
                     torch.empty(E, 2 * I, H // GROUP, **empty)),
         "down": (torch.empty(E, H, I // 2, **empty), torch.empty(E, H, I // GROUP, **empty))}
    for codes, scales in q.values():
        for e in range(E):
            w = normal(codes.shape[1], codes.shape[2] * 2, scale=0.02)
            codes[e], scales[e] = _quantize(w)
    if own:
        import grouped_top_routing_amd as gtr
        st["weights"] = gtr.pack_fp4(*q["gate_up"], *q["down"])
    else:
        st["weights"] = q
        pairs = torch.tensor([_E2M1[c & 7] * (-1 if c & 8 else 1) for b in range(256)
                              for c in (b & 15, b >> 4)], device=DEV)
        st["pairs"] = pairs.view(256, 2)  # a byte's two values
    return st


# ---------------------------------------------------------------------------
# the passes
def run(st):
    return {"select": _select, "select_backward": _select_backward, "balance_loss": _balance_loss,
            "experts": _experts}[st["op"]](st)


def _scores(z, score, like=None):
    """Scores of logits z in the type of `like` (fp32 if none): 0 where z is -inf."""
    z = z.to(like or torch.float32)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _select(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.select(st["logits"], score=st["score"], sel_bias=st["sel_bias"],
                          num_groups=st["groups"], topk_groups=st["topk_groups"],
                          group_best=st["group_best"], topk=st["topk"],
                          renormalize=st["renormalize"])
    # in 64 bits: neighbours in the order may be as close as a rounding
    z = st["logits"].double()
    s = _scores(z, st["score"], torch.float64)
    value = s if st["sel_bias"] is None else s + st["sel_bias"].double()
    value = torch.where(z > -math.inf, value, -math.inf)
    order = z if st["sel_bias"] is None else value
    G = st["groups"]
    if st["topk_groups"] < G:
        T, E = z.shape
        best = value.view(T, G, E // G).sort(2, descending=True).values[:, :, :st["group_best"]]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        total = torch.where(some, total, -math.inf)
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :st["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        order = torch.where(keep.repeat_interleave(E // G, 1), order, -math.inf)
    top, ids = order.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :st["topk"]], ids[:, :st["topk"]]
    w = torch.where(top > -math.inf, s.gather(1, ids), 0.0)
    if st["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(top > -math.inf, ids, -1).to(torch.int32), w.float()


def _select_backward(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.select_backward(st["logits"], st["ids"], st["grad"], score=st["score"],
                                   renormalize=st["renormalize"], load=st["load"],
                                   grad_loss=st["grad_loss"])
    s = _scores(st["logits"], st["score"])
    valid = st["ids"] >= 0
    at = st["ids"].clamp(min=0).long()
    g = torch.where(valid, st["grad"], 0.0)
    w = torch.where(valid, s.gather(1, at), 0.0)
    soft = st["score"] == "softmax"
    if st["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
        each = w * (g - (g * w).sum(1, keepdim=True))
        dz = torch.zeros_like(s).scatter_add_(1, at, each)
        if not soft:
            dz = dz * (1 - s)
    else:
        dz = torch.zeros_like(s).scatter_add_(1, at, g)
        dz = s * (dz - (g * w).sum(1, keepdim=True)) if soft else s * (1 - s) * dz
    if st["load"] is not None:
        q = s if soft else s / s.sum(1, keepdim=True).clamp(min=1e-30)
        d = q * (st["load"] - (q * st["load"]).sum(1, keepdim=True))
        if not soft:
            d = d * (1 - s)
        dz = dz + torch.where(valid.any(1, keepdim=True), st["grad_loss"] * d, 0.0)
    return dz.to(st["logits"].dtype)


def _balance_loss(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.balance_loss(st["logits"], st["ids"], score=st["score"], coef=COEF)
    s = _scores(st["logits"], st["score"])
    q = s if st["score"] == "softmax" else s / s.sum(1, keepdim=True).clamp(min=1e-30)
    valid = st["ids"] >= 0
    rows = valid.any(1)
    T = rows.sum().clamp(min=1)
    E = s.shape[1]
    each = torch.zeros(E + 1, device=s.device)
    each.scatter_add_(0, torch.where(valid, st["ids"], E).long().reshape(-1),
                      torch.ones(valid.numel(), device=s.device))
    share = each[:E] * E / each[:E].sum().clamp(min=1)
    load = COEF * share / T
    return (load * torch.where(rows[:, None], q, 0.0).sum(0)).sum(), load


def _experts(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.expert_ffn_fp4(st["x"], st["src"], st["offsets"], st["weights"],
                                  topk=st["topk"])
    I, bounds, pairs = st["inter"], st["bounds"], st["pairs"]

    def dense(name, e):
        codes, scales = st["weights"][name]
        w = pairs[codes[e].int()].view(codes.shape[1], -1, GROUP)
        return (w * torch.exp2(scales[e].float() - 127.0)[:, :, None]).view(codes.shape[1], -1)

    x = st["x"].float()
    token = (st["src"] // st["topk"]).long()
    y = torch.empty(len(token), x.shape[1], dtype=torch.bfloat16, device=x.device)
    for e in range(BLOCK_EXPERTS):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        gu = x[token[a:b]] @ dense("gate_up", e).t()
        gate, up = gu[:, :I], gu[:, I:]
        h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)  # the operator's h is bf16
        y[a:b] = (h.float() @ dense("down", e).t()).to(torch.bfloat16)
    return y


# ---------------------------------------------------------------------------
# the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"select": _exact_select, "select_backward": _exact_select_backward,
            "balance_loss": _exact_balance, "experts": _exact_experts}[case["op"]](st)


def _log_scores(z, score):
    """Logarithms of the scores, fp64."""
    z = z.double()
    if score == "sigmoid":
        return -torch.log1p(torch.exp(-z.abs())) + z.clamp(max=0.0)
    return z - torch.logsumexp(z, 1, keepdim=True)


def _exact_select(st):
    z = st["logits"].double()
    T, E = z.shape
    s = torch.exp(_log_scores(z, st["score"]))
    out = z == -math.inf
    value = s if st["sel_bias"] is None else s + st["sel_bias"].double()
    order = (z if st["sel_bias"] is None else value).masked_fill(out, -math.inf)
    value = value.masked_fill(out, -math.inf)
    G = st["groups"]
    rows = torch.arange(T, device=z.device)
    # group by group: the best values, one after the other
    left, total = value.view(T, G, E // G).clone(), torch.zeros(T, G, dtype=torch.float64,
                                                                device=z.device)
    none = left.amax(2) == -math.inf
    for _ in range(st["group_best"]):
        best, at = left.max(2)
        total += torch.where(best == -math.inf, 0.0, best)
        left.scatter_(2, at[:, :, None], -math.inf)
    total = total.masked_fill(none, -math.inf)
    rank = ((total[:, None, :] > total[:, :, None])
            | ((total[:, None, :] == total[:, :, None])
               & (torch.arange(G, device=z.device)[None, :] < torch.arange(G, device=z.device)[:, None]))
            ).sum(2)
    order = order.masked_fill((rank >= st["topk_groups"]).repeat_interleave(E // G, 1), -math.inf)
    ids, w = [], []
    place = torch.arange(E, device=z.device)
    for _ in range(st["topk"]):
        best = order.amax(1)
        at = torch.where(order == best[:, None], place, E).amin(1)  # the lowest of equals
        some = best > -math.inf
        ids.append(torch.where(some, at, -1))
        w.append(torch.where(some, s[rows, at], 0.0))
        order[rows, at] = -math.inf
    w = torch.stack(w, 1)
    if st["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.stack(ids, 1).to(torch.int32), w


def _exact_select_backward(st):
    """By the chain rule, slot by slot: w is a function of the scores, and those of z."""
    z = st["logits"].double()
    T, E = z.shape
    s = torch.exp(_log_scores(z, st["score"])).nan_to_num(0.0)
    ds = torch.zeros_like(s)  # gradient with respect to the scores
    chosen = torch.zeros(T, dtype=torch.float64, device=z.device)
    k = st["ids"].shape[1]
    rows = [(st["ids"][:, j] >= 0).nonzero()[:, 0] for j in range(k)]
    cols = [st["ids"][r, j].long() for j, r in enumerate(rows)]
    g = st["grad"].double()
    if st["renormalize"]:
        for r, e in zip(rows, cols):
            chosen[r] += s[r, e]
        inner = torch.zeros_like(chosen)
        for j, (r, e) in enumerate(zip(rows, cols)):
            inner[r] += g[r, j] * s[r, e]
        for j, (r, e) in enumerate(zip(rows, cols)):
            ds[r, e] += torch.where(chosen[r] > 0, g[r, j] / chosen[r]
                                    - inner[r] / chosen[r] ** 2, 0.0)
    else:
        for j, (r, e) in enumerate(zip(rows, cols)):
            ds[r, e] += g[r, j]
    if st["load"] is not None:
        real = (st["ids"] >= 0).any(1)
        c = st["load"].double() * st["grad_loss"].double()
        total = s.sum(1, keepdim=True)  # one, for the softmax
        if st["score"] == "softmax":
            ds[real] += c
        else:
            q = s / total.clamp(min=1e-300)
            ds[real] += ((c - (q * c).sum(1, keepdim=True)) / total.clamp(min=1e-300))[real]
    if st["score"] == "sigmoid":
        return ds * s * torch.exp(_log_scores(-z, "sigmoid"))
    return s * (ds - (s * ds).sum(1, keepdim=True))


def _exact_balance(st):
    s = torch.exp(_log_scores(st["logits"], st["score"])).nan_to_num(0.0)
    if st["score"] == "sigmoid":
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    E = s.shape[1]
    ids = st["ids"].reshape(-1).long()
    count = torch.bincount(ids[ids >= 0], minlength=E).double()
    real = (st["ids"] >= 0).any(1)
    share = E * count / count.sum().clamp(min=1)
    mean = s[real].sum(0) / real.sum().clamp(min=1)
    return COEF * (share * mean).sum(), COEF * share / real.sum().clamp(min=1)


def _exact_experts(st):
    I, k = st["inter"], st["topk"]
    table = torch.tensor([*_E2M1, *(-v for v in _E2M1)], dtype=torch.float64, device=DEV)

    def matrix(name, e):
        codes, scales = st["weights"][name]
        both = torch.stack((codes[e] & 15, codes[e] >> 4), 2).view(codes.shape[1], -1)
        step = torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), scales[e].int() - 127)
        return table[both.long()] * step.repeat_interleave(GROUP, 1)

    y = torch.zeros(len(st["src"]), st["hidden"], dtype=torch.float64, device=DEV)
    row_expert = torch.bucketize(torch.arange(len(y), device=DEV), st["offsets"][1:].long(),
                                 right=True)
    for e in row_expert.unique().tolist():
        at = (row_expert == e).nonzero()[:, 0]
        x = st["x"][(st["src"][at] // k).long()].double()
        both = matrix("gate_up", e)
        gate = x @ both[:I].t()
        h = gate * torch.sigmoid(gate) * (x @ both[I:].t())
        y[at] = h.to(torch.bfloat16).double() @ matrix("down", e).t()
    return y
