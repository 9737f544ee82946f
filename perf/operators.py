"""Cases for timing and checking the training operators of the MoE block.

Three groups of operators:

* rows: tokens sorted by expert (``dispatch``), the gradient of that
  (``dispatch_backward``) and the gradient of the weighted way back
  (``combine_backward``);
* route: the gradient of the router, from the gradient of the combine weights
  to those of the router weights and of the hidden state (``route_backward``);
* adamw: one AdamW step over a list of tensors, with 32-bit states or 8-bit
  ones.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
with the library's calls; ``exact`` computes the same from the definitions in
64 bits.

Routing notation: pair p = t*k + j is slot j of token t; perm_dst[p] is its row
in expert-major order, -1 for a dropped pair (an id that names no expert).
"""
import math

import torch

own = False

EXPERTS = 256
DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# AdamW: hyperparameters of an adapter fine-tune; the step is one in mid-run
LR, BETA1, BETA2, EPS, DECAY, STEP = 2e-5, 0.9, 0.999, 1e-8, 0.01, 100
GRAD_SCALE = 0.5
BLOCK = 32  # elements per scale of an 8-bit state


# ---------------------------------------------------------------------------
# cases
def listed():
    rows = dict(topk=8, hidden=5120, dtype="bf16", weighted=False, dropped=0.0, skew=False)
    route = dict(op="route_backward", hidden=5120, topk=8, renormalize=True, add=True,
                 accumulate=False, skew=False)
    return [
        # a decode batch of the block: latency
        dict(rows, name="dispatch_decode", op="dispatch", tokens=32),
        # a prefill chunk
        dict(rows, name="dispatch_prefill", op="dispatch", tokens=4096),
        # fp32 rows of odd length, weights applied on the way in, replayed ids with holes
        dict(rows, name="dispatch_weighted_odd", op="dispatch", tokens=1537, hidden=1023, topk=5,
             dtype="fp32", weighted=True, dropped=0.03),
        # a training micro-batch
        dict(rows, name="dispatch_grad_micro", op="dispatch_backward", tokens=5120),
        # bf16 rows whose length no 16-byte load divides, with the weights' gradient
        dict(rows, name="dispatch_grad_odd", op="dispatch_backward", tokens=509, hidden=777,
             weighted=True, dropped=0.02),
        # a small fp32 model
        dict(rows, name="combine_grad_small", op="combine_backward", tokens=64, hidden=512,
             dtype="fp32"),
        # the skewed 16K-token batch: the largest
        dict(rows, name="combine_grad_skew", op="combine_backward", tokens=16384, skew=True),
        # the router's gradient: a decode-sized batch and a skewed training micro-batch
        dict(route, name="route_grad_decode", tokens=32),
        dict(route, name="route_grad_micro", tokens=5120, skew=True),
        # the router's weights alone, in fp32
        dict(name="adamw_router", op="adamw", layout="ragged", total=256 * 5120, count=1, mix=0,
             params="fp32", bits=32),
        # one layer's rank-16 expert adapters: bf16 with fp32 masters
        dict(name="adamw_adapters", op="adamw", layout="adapters", experts=256, hidden=5120,
             inter=2560, rank=16, params="bf16", bits=32),
        dict(name="adamw_adapters_8bit", op="adamw", layout="adapters", experts=256, hidden=5120,
             inter=2560, rank=16, params="bf16", bits=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_backward", "combine_backward", "route_backward",
                     "adamw"])
    if op == "adamw":
        return dict(op=op, layout="ragged", total=_log(rng, 1000, 60_000_000),
                    count=_log(rng, 1, 200), mix=rng.randrange(1 << 16),
                    params=rng.choice(["fp32", "bf16"]), bits=rng.choice([32, 8]))
    if op == "route_backward":
        return dict(op=op, tokens=_log(rng, 1, 5120), hidden=256 * rng.randint(1, 24),
                    topk=rng.randint(1, 8), renormalize=rng.random() < 0.7,
                    add=rng.random() < 0.5, accumulate=rng.random() < 0.5,
                    skew=rng.random() < 0.5)
    hidden = _log(rng, 8, 7168)
    if rng.random() < 0.5:
        hidden = max(8, hidden // 8 * 8)
    dtype, topk = rng.choice(["bf16", "fp32"]), rng.randint(1, 8)
    most = 16384 * 8 * 5120 * 2 // (hidden * topk * (2 if dtype == "bf16" else 4))
    weighted = rng.random() < 0.5
    return dict(op=op, tokens=_log(rng, 1, min(16384, most)), hidden=hidden, topk=topk,
                dtype=dtype, weighted=weighted, dropped=rng.choice([0.0, 0.0, 0.05]),
                skew=rng.random() < 0.5)


def _sizes(case):
    """Element counts of the tensors of an adamw case."""
    if case["layout"] == "adapters":
        e, h, i, r = case["experts"], case["hidden"], case["inter"], case["rank"]
        return [e * r * h, e * 2 * i * r, e * r * i, e * h * r]
    count, left = case["count"], case["total"]
    parts, x = [], case["mix"] + 1
    for _ in range(count):
        x = (x * 1103515245 + 12345) % (1 << 31)
        parts.append(1 + x % 1000)
    return [max(1, left * q // sum(parts)) for q in parts]


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        param = 8 + 4 if case["params"] == "fp32" else 8 + 2 + 2
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (param + state), "flops": 16 * n}
    T, H, k = case["tokens"], case["hidden"], case["topk"]
    if case["op"] == "route_backward":
        w = EXPERTS * H * 4
        return {"bytes": T * H * 2 * (3 if case["add"] else 2)
                + w * (3 if case["accumulate"] else 2) + 16 * T * k, "flops": 4 * T * k * H}
    s = 2 if case["dtype"] == "bf16" else 4
    n = T * k * (1 - case["dropped"])
    one, many = T * H * s, n * H * s
    if case["op"] == "dispatch":
        return {"bytes": one + many + 4 * T * k * (2 if case["weighted"] else 1),
                "flops": n * H if case["weighted"] else 0}
    if case["op"] == "dispatch_backward":
        return {"bytes": one * (2 if case["weighted"] else 1) + many
                + 4 * T * k * (3 if case["weighted"] else 1),
                "flops": n * H * (4 if case["weighted"] else 1)}
    return {"bytes": one + 2 * many + 12 * T * k, "flops": 3 * n * H}


# ---------------------------------------------------------------------------
# inputs
def _routing(case, g):
    """Expert ids [T, k] and the permutation they give."""
    T, k = case["tokens"], case["topk"]
    score = -torch.log(-torch.log(torch.rand(T, EXPERTS, generator=g, device=DEV).clamp_(1e-9, 1 - 1e-6)))
    if case["skew"]:  # sixteen experts take most of the tokens
        score[:, 5::16] += 4.0
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    if case.get("dropped"):
        ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < case["dropped"], -1, ids)
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, EXPERTS, flat)
    src = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=EXPERTS + 1)[:EXPERTS]
    offsets = torch.zeros(EXPERTS + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    dst = torch.empty_like(src)
    dst[src] = torch.arange(T * k, device=DEV)
    dst = torch.where(flat < 0, -1, dst)
    return ids, offsets, src.to(torch.int32), dst.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)

    st = dict(case)
    if case["op"] == "adamw":
        return _prepare_adamw(case, st, normal, seed)
    T, H, k = case["tokens"], case["hidden"], case["topk"]
    ids, offsets, src, dst = _routing(case, g)
    if case["op"] == "route_backward":
        st.update(ids=ids, offsets=offsets, src=src, x=normal(T, H, dtype=torch.bfloat16),
                  w=normal(EXPERTS, H, scale=0.02), logits=normal(T, k, scale=1.5) + 1.0,
                  grad=normal(T, k, scale=1e-2),
                  add_to=normal(T, H, scale=1e-3, dtype=torch.bfloat16) if case["add"] else None,
                  # accumulated gradients start from an earlier micro-batch's
                  acc=normal(EXPERTS, H, scale=0.1) if case["accumulate"] else None)
        return st
    dt = _TYPES[case["dtype"]]
    st.update(dst=dst, weights=torch.rand(T, k, generator=g, device=DEV) / k)
    # the sorted rows' buffer: rows that no pair names keep their zeros (the
    # plain form scatters dropped pairs into the spare last row)
    st["buffer"] = torch.zeros(T * k + 1, H, dtype=dt, device=DEV)
    if case["op"] == "dispatch":
        st["x"] = normal(T, H, dtype=dt)
    elif case["op"] == "dispatch_backward":
        st.update(x=normal(T, H, dtype=dt), grad=normal(T * k, H, dtype=dt))
    else:
        st.update(grad=normal(T, H, dtype=dt), y=normal(T * k, H, dtype=dt))
    return st


def _prepare_adamw(case, st, normal, seed):
    sizes = _sizes(case)
    starts, total = [], 0
    for n in sizes:  # the tensors lie in flat buffers, each at a multiple of 32 elements
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK

    def views(flat, per=1):
        return [flat[a // per:a // per + -(-n // per)] for a, n in zip(starts, sizes)]

    lengths = torch.tensor(sizes, device=DEV)
    which = torch.repeat_interleave(torch.arange(len(sizes), device=DEV),
                                    (lengths + BLOCK - 1) // BLOCK * BLOCK, output_size=total)
    place = torch.arange(total, device=DEV) - torch.tensor(starts, device=DEV)[which]
    used = (place < lengths[which]).float()
    low = case["params"] == "bf16"
    # gradients of blocks differ in size, as those of experts that see few or many tokens do
    size = 1e-3 * torch.exp(normal(total // BLOCK)).repeat_interleave(BLOCK) * used
    master = normal(total, scale=0.02) * used
    grad = (normal(total) * size).to(torch.bfloat16 if low else torch.float32)
    m = normal(total, scale=0.3) * size
    root = (0.5 + normal(total).abs()) * size
    param = master.to(torch.bfloat16) if low else master
    flat = dict(param=param, master=master if low else None)
    if case["bits"] == 32:
        flat.update(m=m, v=root * root, m_scale=None, v_scale=None)
    else:
        for name, x in (("m", m), ("v", root)):
            code = _scale_code(x.abs().view(-1, BLOCK).amax(1))
            flat[name + "_scale"] = code.to(torch.uint8).view(torch.float8_e8m0fnu)
            flat[name] = (x.view(-1, BLOCK) * _inverse(code)[:, None]).view(-1).to(torch.float8_e4m3fn)
    st.update(flat=flat, grad=grad, seed=seed % 65521, place=place, which=which)
    if own:
        import grouped_top_routing_amd as gtr
        state = {"exp_avg": views(flat["m"]), "exp_avg_sq": views(flat["v"])}
        if low:
            state["master"] = views(master)
        if case["bits"] == 8:
            state["exp_avg_scale"] = views(flat["m_scale"], BLOCK)
            state["exp_avg_sq_scale"] = views(flat["v_scale"], BLOCK)
        st["opt"] = gtr.AdamW(views(param), lr=LR, betas=(BETA1, BETA2), eps=EPS,
                              weight_decay=DECAY, state_bits=case["bits"], seed=st["seed"],
                              state=state, step_count=STEP - 1)
        st["grads"] = views(grad)
    else:
        st["step"] = STEP - 1
    return st


# ---------------------------------------------------------------------------
# the passes
def run(st):
    return {"dispatch": _dispatch, "dispatch_backward": _dispatch_backward,
            "combine_backward": _combine_backward, "route_backward": _route_backward,
            "adamw": _adamw}[st["op"]](st)


def _dispatch(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.dispatch(st["x"], st["dst"], topk=st["topk"],
                            topk_w=st["weights"] if st["weighted"] else None,
                            out=st["buffer"][:-1])
    x, buf = st["x"], st["buffer"]
    rows = x[:, None, :].expand(-1, st["topk"], -1)
    if st["weighted"]:
        rows = (rows.float() * st["weights"][:, :, None]).to(x.dtype)
    buf[_spare(st["dst"], buf)] = rows.reshape(-1, x.shape[1])
    return buf[:-1]


def _spare(dst, buf):
    return torch.where(dst < 0, buf.shape[0] - 1, dst).long()


def _dispatch_backward(st):
    if own:
        import grouped_top_routing_amd as gtr
        if st["weighted"]:
            return gtr.dispatch_backward(st["grad"], st["dst"], topk=st["topk"], x=st["x"],
                                         topk_w=st["weights"])
        return gtr.dispatch_backward(st["grad"], st["dst"], topk=st["topk"])
    T, k = st["x"].shape[0], st["topk"]
    rows = st["grad"][st["dst"].clamp(min=0).long()].float()
    rows = torch.where((st["dst"] >= 0)[:, None], rows, 0.0).view(T, k, -1)
    if not st["weighted"]:
        return rows.sum(1).to(st["grad"].dtype)
    grad_w = (rows * st["x"].float()[:, None, :]).sum(2)
    return (rows * st["weights"][:, :, None]).sum(1).to(st["grad"].dtype), grad_w


def _combine_backward(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.combine_backward(st["grad"], st["y"], st["dst"], st["weights"],
                                    routed_scaling=2.5, out=st["buffer"][:-1])
    g, buf = st["grad"].float(), st["buffer"]
    T, k = st["weights"].shape
    rows = st["y"][st["dst"].clamp(min=0).long()].float().view(T, k, -1)
    grad_w = torch.where(st["dst"].view(T, k) >= 0, 2.5 * (rows * g[:, None, :]).sum(2), 0.0)
    grad_y = ((2.5 * st["weights"])[:, :, None] * g[:, None, :]).to(buf.dtype)
    buf[_spare(st["dst"], buf)] = grad_y.view(T * k, -1)
    return buf[:-1], grad_w


def _route_backward(st):
    if own:
        import grouped_top_routing_amd as gtr
        return gtr.route_backward(st["x"], st["w"], st["ids"], st["logits"], st["grad"],
                                  st["src"], st["offsets"], renormalize=st["renormalize"],
                                  grad_x_add=st["add_to"], grad_w_router=st["acc"])
    ids, z, g = st["ids"].long(), st["logits"], st["grad"]
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    if st["renormalize"]:
        w = s / s.sum(1, keepdim=True)
        dz = w * rest * (g - (g * w).sum(1, keepdim=True))
    else:
        dz = s * rest * g
    dense = torch.zeros(z.shape[0], EXPERTS, device=z.device).scatter_add_(1, ids, dz)
    grad_w = dense.t() @ st["x"].float()
    if st["accumulate"]:
        grad_w = st["acc"].add_(grad_w)
    grad_x = dense @ st["w"]
    if st["add"]:
        grad_x = st["add_to"].float() + grad_x
    return grad_w, grad_x.to(torch.bfloat16)


def _mix(z):
    """Scrambles 32-bit words (held in int64)."""
    z = ((z ^ (z >> 16)) * 0x7A3D5E4B) & 0xFFFFFFFF
    z = ((z ^ (z >> 15)) * 0xB5297A4D) & 0xFFFFFFFF
    return z ^ (z >> 16)


def _random(place, which, seed, step):
    """32 random bits per element of an 8-bit state, from the seed, the step,
    the tensor's place in the list and the element's place in the tensor."""
    key = _mix((seed * 0x9E3779B9 + step * 0x85157AF5 + which * 0x632BE5AB) & 0xFFFFFFFF)
    return _mix(((place * 0x9E3779B1) & 0xFFFFFFFF) ^ key)


def _scale_code(most):
    """E8M0 code of the least power of two by which `most` is at most 448, the
    largest E4M3 value (at least 2^-126)."""
    u = most.view(torch.int32)
    return ((u >> 23) - 8 + ((u & 0x7FFFFF) > 0x600000)).clamp(min=1)


def _inverse(code):
    return ((254 - code) << 23).view(torch.float32)


def _pack(x, random, low):
    """E4M3 codes of x (|x| at most 448), rounded up or down by 16 random bits."""
    y = x.abs()
    big = ((y.view(torch.int32) + (random << 4).to(torch.int32)) >> 20) - 960
    small = torch.floor(y * 512.0 + random.float() * 2.0 ** -16).to(torch.int32)
    code = torch.where(y >= 2.0 ** -6, big, small).clamp(max=126)
    if low:  # not zero where the value is not
        code = torch.where(x > 0, code.clamp(min=1), code)
    return torch.where(x < 0, code + 128, code).to(torch.uint8).view(torch.float8_e4m3fn)


def _adamw(st):
    flat = st["flat"]
    names = [n for n in ("param", "master", "m", "v", "m_scale", "v_scale") if flat[n] is not None]
    if own:
        st["opt"].step(st["grads"], grad_scale=GRAD_SCALE)
        return {n: flat[n] for n in names}
    st["step"] += 1
    t = st["step"]
    g = st["grad"].float() * GRAD_SCALE
    p = flat["param"] if flat["master"] is None else flat["master"]
    if st["bits"] == 32:
        m, v = flat["m"], flat["v"]
    else:
        m = (flat["m"].float().view(-1, BLOCK) * flat["m_scale"].float()[:, None]).view(-1)
        v = (flat["v"].float().view(-1, BLOCK) * flat["v_scale"].float()[:, None]).view(-1)
        v = v * v
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = v.sqrt()
    update = m / (root * (1 / math.sqrt(1 - BETA2 ** t)) + EPS)
    p.copy_(p * (1 - LR * DECAY) - update * (LR / (1 - BETA1 ** t)))
    if flat["master"] is not None:
        flat["param"].copy_(p)
    if st["bits"] == 32:
        flat["m"].copy_(m)
        flat["v"].copy_(v)
        return {n: flat[n] for n in names}
    random = _random(st["place"], st["which"], st["seed"], t)
    for name, x, bits, low in (("m", m, random & 0xFFFF, False), ("v", root, random >> 16, True)):
        code = _scale_code(x.abs().view(-1, BLOCK).amax(1))
        y = (x.view(-1, BLOCK) * _inverse(code)[:, None]).view(-1)
        flat[name].copy_(_pack(y, bits, low))
        flat[name + "_scale"].copy_(code.to(torch.uint8).view(torch.float8_e8m0fnu))
    return {n: flat[n] for n in names}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(st)
    if case["op"] == "route_backward":
        return _exact_route(st)
    T, k = case["tokens"], case["topk"]
    dst = st["dst"].view(T, k)
    w = st["weights"].double()
    if case["op"] == "dispatch":
        out = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device=DEV)
        for j in range(k):
            at = (dst[:, j] >= 0).nonzero()[:, 0]
            x = st["x"][at].double()
            out[dst[at, j].long()] = x * w[at, j][:, None] if case["weighted"] else x
        return out
    g = st["grad"]
    grad_w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    if case["op"] == "dispatch_backward":
        out = torch.zeros(T, case["hidden"], dtype=torch.float64, device=DEV)
        for j in range(k):
            at = (dst[:, j] >= 0).nonzero()[:, 0]
            row = g[dst[at, j].long()].double()
            grad_w[at, j] = (row * st["x"][at].double()).sum(1)
            out[at] += row * w[at, j][:, None] if case["weighted"] else row
        return (out, grad_w) if case["weighted"] else out
    out = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device=DEV)
    for j in range(k):
        at = (dst[:, j] >= 0).nonzero()[:, 0]
        row, gt = dst[at, j].long(), g[at].double()
        grad_w[at, j] = 2.5 * (gt * st["y"][row].double()).sum(1)
        out[row] = 2.5 * w[at, j][:, None] * gt
    return out, grad_w


def _exact_route(st):
    z, g = st["logits"].double(), st["grad"].double()
    T, k = z.shape
    s = 1 / (1 + torch.exp(-z))
    total = s.sum(1)
    x, W = st["x"].double(), st["w"].double()
    grad_w = st["acc"].double() if st["accumulate"] else torch.zeros_like(W)
    grad_x = st["add_to"].double() if st["add"] else torch.zeros_like(x)
    for j in range(k):
        if st["renormalize"]:  # d(s_i / total) / d s_j
            ds = g[:, j] / total - (g * s).sum(1) / total ** 2
        else:
            ds = g[:, j]
        dz = ds * s[:, j] / (1 + torch.exp(z[:, j]))
        e = st["ids"][:, j].long()
        grad_x = grad_x + dz[:, None] * W[e]
        grad_w = grad_w.index_add(0, e, dz[:, None] * x)
    return grad_w, grad_x


def _exact_adamw(st):
    flat = st["flat"]
    g = st["grad"].double() * GRAD_SCALE
    p = (flat["param"] if flat["master"] is None else flat["master"]).double()
    if st["bits"] == 32:
        m, v = flat["m"].double(), flat["v"].double()
    else:
        m = flat["m"].double() * flat["m_scale"].double().repeat_interleave(BLOCK)
        v = (flat["v"].double() * flat["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    hat = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
    p = p - LR * DECAY * p - LR * hat
    out = {"param": p}
    if flat["master"] is not None:
        out["master"] = p
    if st["bits"] == 32:
        return dict(out, m=m, v=v)
    random = _random(st["place"], st["which"], st["seed"], STEP)
    for name, x, bits in (("m", m, random & 0xFFFF), ("v", v.sqrt(), random >> 16)):
        most, exponent = torch.frexp(x.abs().view(-1, BLOCK).amax(1))
        scale = torch.exp2((exponent - 9 + (most > 0.875).int()).clamp(min=-126).double())
        y = (x.view(-1, BLOCK) / scale[:, None]).view(-1)
        step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
        q = torch.floor(y.abs() / step + bits.double() / 65536) * step
        if name == "v":
            q = torch.where(y > 0, q.clamp(min=2.0 ** -9), q)
        out[name] = q * torch.sign(y)
        out[name + "_scale"] = scale
    return out
