"""The calls on the GPU where they are easiest to get wrong: scratch memory of
captured calls, steps counted per tensor, weight decay far below a rounding,
batches at the edges of a kernel's loops and grids, and the forms that
RouterTrainer can be built in.

Bounds count roundings as those of test_gpu_train.py do; U is half a step of
fp32."""
import copy
import ctypes
import weakref

import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
import synth
from grouped_top_routing_amd import _lib
from oracle import train
from parity_util import say
from test_gpu_train import (BF, DEV, F, HP, NAMES, U, _adam_bounds, _opt, _route_bounds,
                            _router_case, n64, rows, u_of, weights, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# scratch memory of captured calls
def _route_inputs(T, seed):
    d = synth.make_inputs(synth.workload("tiny", T=T), seed, device=DEV)
    return d["x"], d["w_router"]


def test_captured_calls_leave_the_default_workspace_alone():
    """A graph captured on a stream whose default workspace exists must not
    hold that workspace: it may grow (and be given back to the allocator) while
    the graph lives, and another graph captured on the stream would share it."""
    say("[workspace] captured route and the stream's default workspace")
    x, W = _route_inputs(300, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = gtr.route(x, W, return_logits=True)
    torch.cuda.synchronize()
    buf = _lib._default_ws[(x.device, stream.cuda_stream)]._buf
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = gtr.route(x, W, return_logits=True)
    for _ in range(3):
        buf.fill_(0x5A)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((buf == 0x5A).all())


def test_two_graphs_captured_on_one_stream_replay_at_once():
    say("[workspace] two graphs of the forward stages, captured on one stream")
    cases = [_route_inputs(900, s) for s in (1, 2)]
    d = synth.make_inputs("tiny", 0, device=DEV)
    gu, dn = d["w_gate_up"], d["w_down"]

    def chain(x, W):
        ids, w, z = gtr.route(x, W, return_logits=True)
        _, off, src, dst = gtr.permute(ids)
        return ids, w, z, gtr.combine(gtr.expert_ffn(x, src, off, gu, dn), dst, w)

    want = [chain(*c) for c in cases]
    torch.cuda.synchronize()
    graphs, got, stream = [], [], torch.cuda.Stream()
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            got.append(chain(*c))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for outs in got:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for outs, ref in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_a_captured_workspace_outlives_its_growth():
    say("[workspace] the buffer a graph holds is kept when the workspace grows")
    x, W = _route_inputs(200, 3)
    big, _ = _route_inputs(6000, 4)
    ws = gtr.Workspace()
    want = gtr.route(x, W, workspace=ws)
    want_big = gtr.route(big, W)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gtr.route(x, W, workspace=ws)
    held = weakref.ref(ws._buf)
    got_big = gtr.route(big, W, workspace=ws)
    assert ws._buf is not held() and held() is not None
    for _ in range(3):
        got[0].zero_(), got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(gtr.route(big, W, workspace=ws), want_big))
    assert all(torch.equal(a, b) for a, b in zip(got_big, want_big))


# ---------------------------------------------------------------------------
# AdamW counts the steps of each tensor
LATE_SIZES = (1000, 70, 33, 2049)


def _late_grads(step, dt):
    """Gradients of step 1, 2, ...: always; from the fifth; odd ones; never."""
    on = (True, step >= 5, step % 2 == 1, False)
    return [rows(1, n, dt, 10 * step + i).view(-1) * 0.1 if yes else None
            for i, (n, yes) in enumerate(zip(LATE_SIZES, on))]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("dt", [F, BF], ids=NAMES.get)
def test_adamw_counts_the_steps_of_each_tensor(bits, capturable, dt):
    """A tensor without a gradient makes no step: its bias correction (and the
    rounding of its 8-bit states) goes by the steps it has made."""
    say(f"[adamw] late and rare gradients, {bits} bits, capturable={capturable}, {dt}")
    params = [rows(1, n, dt, i).view(-1) for i, n in enumerate(LATE_SIZES)]
    never = params[3].clone()
    opt = _opt(params, state_bits=bits, seed=11, capturable=capturable)
    made = [0] * 4

    def state(i):
        st = opt.state
        p = n64(st["master"][i] if dt == BF else params[i])
        if bits == 32:
            return p, n64(st["exp_avg"][i]), n64(st["exp_avg_sq"][i])
        m, r = (train.decode_8bit(st[k][i].view(torch.uint8).cpu().numpy(),
                                  st[k + "_scale"][i].view(torch.uint8).cpu().numpy())
                for k in ("exp_avg", "exp_avg_sq"))
        return p, m, r * r

    for step in range(1, 9):
        grads = _late_grads(step, dt)
        before = [state(i) for i in range(4)]
        opt.step(grads)
        for i, g in enumerate(grads):
            if g is None:
                assert all(np.array_equal(a, b) for a, b in zip(state(i), before[i]))
                continue
            made[i] += 1
            p0, m0, v0 = before[i]
            ref = train.adamw(p0, n64(g), m0, v0, step=made[i], **HP)
            bounds = _adam_bounds(p0, n64(g), m0, v0, made[i], 1.0)
            got = state(i)
            within(got[0], ref[0], bounds[0], f"step {step} tensor {i}")
            if bits == 32:
                within(got[1], ref[1], bounds[1], "m")
                within(got[2], ref[2], bounds[2], "v")
                continue
            f32 = np.float32
            root = np.sqrt(v0)  # exact: codes and scales are short
            m, _, root = train.adamw_state_f32(n64(g), m0, f32(root) * f32(root),
                                               beta1=HP["beta1"], beta2=HP["beta2"])
            random = train.rounding_bits(11, made[i], i, len(p0))
            for k, x, b, low in (("exp_avg", m, random & np.uint64(0xFFFF), False),
                                 ("exp_avg_sq", root, random >> np.uint64(16), True)):
                code, scale = train.encode_8bit(x, b, low)
                raw = opt.state[k][i].view(torch.uint8).cpu().numpy()
                assert np.array_equal(train.decode_8bit(raw, scale),
                                      train.decode_8bit(code, scale)), (step, i, k)
    assert torch.equal(params[3], never)
    assert opt.step_count == 8
    assert list(opt.step_counts) == made == [8, 4, 4, 0]


def test_adamw_first_update_of_a_late_tensor_is_the_rate():
    # from zero states the first update is lr sign(g), whatever the others did
    say("[adamw] a first gradient after 500 steps of the others")
    p, q = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    g = torch.ones(64, device=DEV)
    opt = gtr.AdamW([p, q], lr=1e-3, weight_decay=0.0)
    for _ in range(500):
        opt.step([g, None])
    opt.step([None, g])
    # m / (1 - b1) and sqrt(v / (1 - b2)) are 1 within a few roundings; eps is 1e-8
    within(q, np.full(64, -1e-3), 1e-3 * (16 * U + 1e-8) * np.ones(64), "first update")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_adamw_step_counts_continue_from_a_checkpoint(bits, capturable):
    say(f"[adamw] step_count as a list, {bits} bits, capturable={capturable}")
    a_params = [rows(1, n, BF, i).view(-1) for i, n in enumerate(LATE_SIZES)]
    a = _opt(a_params, state_bits=bits, seed=2, capturable=capturable)
    for step in range(1, 6):
        a.step(_late_grads(step, BF))
    counts = a.step_counts
    assert list(counts) == [5, 1, 3, 0]
    state = {k: [None if t is None else t.clone() for t in v] for k, v in a.state.items()}
    b_params = [t.clone() for t in a_params]
    b = _opt(b_params, state_bits=bits, seed=2, state=state, step_count=counts,
             capturable=not capturable)
    assert list(b.step_counts) == [5, 1, 3, 0] and b.step_count == 5
    for step in range(6, 9):
        a.step(_late_grads(step, BF))
        b.step(_late_grads(step, BF))
    for x, y in zip(a_params, b_params):
        assert torch.equal(x, y)
    for k in state:
        for x, y in zip(a.state[k], state[k]):
            assert torch.equal(x.float(), y.float())
    assert list(a.step_counts) == list(b.step_counts) == [8, 4, 4, 0]


def test_adamw_captured_step_without_some_gradients_counts_on():
    say("[adamw] a captured step of some of the tensors, replayed among eager ones")
    def made():
        return [rows(1, n, F, i).view(-1) for i, n in enumerate(LATE_SIZES)]
    for bits in (32, 8):
        pc, pe = made(), made()
        oc = _opt(pc, state_bits=bits, seed=4, capturable=True)
        oe = _opt(pe, state_bits=bits, seed=4)
        every = [rows(1, n, F, 50 + i).view(-1) for i, n in enumerate(LATE_SIZES)]
        some = [g if i % 2 else None for i, g in enumerate(every)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            oc.step(some)
        assert list(oc.step_counts) == [0] * 4
        for i in range(4):
            graph.replay()
            oe.step(some)
            torch.cuda.synchronize()
            for a, b in zip(pc, pe):
                assert torch.equal(a, b), (bits, i)
            oc.step(every)
            oe.step(every)
            for a, b in zip(pc, pe):
                assert torch.equal(a, b), (bits, i)
        assert list(oc.step_counts) == list(oe.step_counts) == [4, 8, 4, 8]
        assert oc.step_count == oe.step_count == 8


def test_adamw_refuses_wrong_step_counts_and_keeps_its_own():
    p, q = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    for bad, what in (([1], "one step count per parameter"), ([1, 2, 3], "one step count per"),
                      ([1, -1], "negative")):
        with pytest.raises(ValueError, match=what):
            gtr.AdamW([p, q], step_count=bad)
    g = torch.ones(64, device=DEV)
    for capturable in (False, True):
        opt = gtr.AdamW([p, q], capturable=capturable)
        opt.step([g, None])
        for bad in (dict(lr=-1.0), dict(grad_scale=float("nan"))):
            with pytest.raises(gtr.MoeError):
                opt.step([g, None], **bad)
            with pytest.raises(gtr.MoeError):
                opt.step([g, g], **bad)
        assert list(opt.step_counts) == [1, 0] and opt.step_count == 1


# ---------------------------------------------------------------------------
# AdamW: decay far below a rounding of the parameter
@pytest.mark.parametrize("lr,wd", [(2e-5, 0.01), (2e-6, 0.01), (1e-4, 0.1), (3e-3, 0.1), (1e-5, 0.0)])
@pytest.mark.parametrize("dt", [F, BF], ids=NAMES.get)
@pytest.mark.parametrize("device_rate", [False, True])
def test_adamw_decay_keeps_its_mean(lr, wd, dt, device_rate):
    """p - lr wd p - ... with lr wd down to 2e-8 (a rounding of p is 6e-8): an
    element cannot show it, the mean over many, whose updates differ, does.

    An element's error is at most e = U |p'| (its one rounding, of either sign)
    + 16 U |update| (of a sign independent of p's), except for decay's own
    factor, product and sum, 3 U lr wd |p|; where lr wd is 2^-12 and more, the
    product with 1 - lr wd adds a rounding of either sign and that factor's own
    error (U / 2) |p|.  By Hoeffding the signed sum of the errors of either
    sign passes 6 sqrt(sum e^2) with a probability of 3e-8."""
    say(f"[adamw] decay lr={lr} wd={wd} {dt} device_rate={device_rate}")
    n = 1 << 20
    g = torch.Generator(device=DEV).manual_seed(7)
    p32 = (torch.rand(n, generator=g, device=DEV) + 0.5) * torch.where(
        torch.rand(n, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    grad = torch.randn(n, generator=g, device=DEV)
    m, root = torch.randn(n, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV) + 0.5
    p = p32.clone() if dt == F else p32.to(BF)
    state = {"exp_avg": [m.clone()], "exp_avg_sq": [root * root],
             "master": [None if dt == F else p32.clone()]}
    opt = gtr.AdamW([p], lr=lr, weight_decay=wd, state=state, step_count=99)
    start = p32.double()
    v0 = (root * root).double()
    rate = torch.full((1,), lr, device=DEV) if device_rate else lr
    lr = float(rate) if device_rate else lr
    opt.step([grad], lr=rate)
    got = (p if dt == F else opt.state["master"][0]).double()
    b1, b2, eps = 0.9, 0.999, 1e-8
    m1 = b1 * m.double() + (1 - b1) * grad.double()
    v1 = b2 * v0 + (1 - b2) * grad.double() ** 2
    upd = lr * (m1 / (1 - b1 ** 100)) / ((v1 / (1 - b2 ** 100)).sqrt() + eps)
    want = start - lr * wd * start - upd
    err = got - want
    large = lr * wd >= 2.0 ** -12
    e = (2 if large else 1) * U * got.abs() + 16 * U * upd.abs()
    factor = lr * wd * 3 * U + (U / 2 if large else 0.0)
    assert bool((err.abs() <= 1.01 * (e + factor * start.abs())).all())
    signed = abs(float((err * start.sign()).sum()))
    allowed = 6 * float((e * e).sum().sqrt()) + factor * float(start.abs().sum())
    whole = lr * wd * float(start.abs().sum())
    say(f"  signed error {signed:.3e}, allowed {allowed:.3e}, decay {whole:.3e}")
    assert signed <= allowed


def test_adamw_infinite_parameters_stay_so():
    say("[adamw] infinite parameters under decay")
    for wd in (0.0, 1e-3, 0.5):
        for bits in (32, 8):
            p = torch.tensor([float("inf"), -float("inf"), 1.0, float("nan")], device=DEV)
            gtr.AdamW([p], lr=1e-2, weight_decay=wd, state_bits=bits).step(
                [torch.tensor([1.0, 1.0, 1.0, 1.0], device=DEV)])
            assert torch.isposinf(p[0]) and torch.isneginf(p[1]) and torch.isnan(p[3])
            assert torch.isfinite(p[2])


# ---------------------------------------------------------------------------
# AdamW beside autograd
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_state_of_parameters_that_require_grad(bits):
    say(f"[adamw] nn.Parameter, {bits} bits")
    params = [torch.nn.Parameter(rows(1, 100, dt, 1).view(-1)) for dt in (BF, F)]
    opt = _opt(params, state_bits=bits)
    for k, v in opt.state.items():
        assert all(t is None or (not t.requires_grad and t.grad_fn is None) for t in v), k
    saved = copy.deepcopy(opt.state)
    assert torch.equal(saved["master"][0], params[0].detach().float())
    grads = [rows(1, 100, p.dtype, 2).view(-1) for p in params]
    opt.step(grads)
    assert torch.equal(params[0].detach(), opt.state["master"][0].to(BF))
    assert not torch.equal(saved["master"][0], opt.state["master"][0])


def test_adamw_tells_autograd_that_parameters_changed():
    say("[adamw] a backward pass through parameters that a step has changed since")
    for dt in (F, BF):
        p = torch.nn.Parameter(rows(1, 64, dt, 3).view(-1))
        q = torch.nn.Parameter(rows(1, 64, dt, 4).view(-1))
        opt = _opt([p, q])
        loss_p, loss_q = (p * p).sum(), (q * q).sum()
        opt.step([torch.ones(64, dtype=dt, device=DEV), None])
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss_p.backward()
        loss_q.backward()  # q had no gradient and stayed
        assert torch.equal(q.grad, 2 * q.detach())


def test_adamw_refuses_memory_that_overlaps():
    say("[adamw] parameters and states that share memory")
    b = torch.zeros(256, device=DEV)
    for params in ([b[:64], b[32:96]], [b, b[128:192]], [b[128:192], b[64:200]],
                   [b[:64], b.view(BF)[64:72]]):
        with pytest.raises(ValueError, match="overlap"):
            gtr.AdamW(params)
    gtr.AdamW([b[:64], b[64:128], b[128:128], b[128:]])  # side by side
    p, m, v = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    for state in ({"exp_avg": [m], "exp_avg_sq": [m]}, {"exp_avg": [p], "exp_avg_sq": [v]}):
        with pytest.raises(ValueError, match="overlap"):
            gtr.AdamW([p], state=state)
    gtr.AdamW([p], state={"exp_avg": [m], "exp_avg_sq": [v]})
    low = torch.zeros(64, dtype=BF, device=DEV)
    codes = torch.zeros(128, dtype=torch.uint8, device=DEV)
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    state = {"master": [p], "exp_avg": [codes[:64].view(f8)], "exp_avg_sq": [codes[64:].view(f8)],
             "exp_avg_scale": [torch.zeros(2, dtype=torch.uint8, device=DEV).view(e8)],
             "exp_avg_sq_scale": [torch.zeros(2, dtype=torch.uint8, device=DEV).view(e8)]}
    gtr.AdamW([low], state=state, state_bits=8)
    state["exp_avg_sq_scale"] = [codes[126:].view(e8)]
    with pytest.raises(ValueError, match="overlap"):
        gtr.AdamW([low], state=state, state_bits=8)


# ---------------------------------------------------------------------------
# rows and the router's gradient
def test_row_calls_refuse_outputs_that_overlap_inputs():
    say("[rows] out= that shares memory with an input")
    T, H, k = 64, 128, 2
    buf = torch.zeros(2 * T * k * H, device=DEV)
    x, apart = buf[:T * H].view(T, H), buf[T * H:T * H + T * k * H].view(T * k, H)
    dst = torch.arange(T * k, dtype=torch.int32, device=DEV)
    w = torch.ones(T, k, device=DEV)
    for start in (0, T * H - 4):
        with pytest.raises(gtr.MoeError):
            gtr.dispatch(x, dst, topk=k, out=buf[start:start + T * k * H].view(T * k, H))
    gtr.dispatch(x, dst, topk=k, out=apart)  # side by side
    with pytest.raises(gtr.MoeError):
        gtr.combine_backward(x, apart, dst, w, out=apart)
    with pytest.raises(gtr.MoeError):
        gtr.combine_backward(x, None, dst, w, need_grad_w=False,
                             out=buf[:T * k * H].view(T * k, H))
    xb, W, ids, z, g, src, off, _ = _router_case(40, 256, 8, 1)
    with pytest.raises(gtr.MoeError):
        gtr.route_backward(xb, W, ids, z, g, src, off, grad_w_router=W)
    assert float(buf.abs().max()) == 0


def test_route_backward_past_2_to_34():
    """2^24 + 5 tokens of 256 columns (a limit that counted workgroups which
    only batches below 4096 tokens launch refused it); row offsets pass 2^32
    elements.  With one slot and no renormalisation every gradient is one
    product: grad x rows are checked singly, grad W against sums in fp64."""
    T, H = (1 << 24) + 5, 256
    say(f"[route_backward] {T} tokens of {H} columns")
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(T, H, generator=g, device=DEV, dtype=BF)
    W = 0.02 * torch.randn(256, H, generator=g, device=DEV)
    ids = torch.randint(0, 256, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    z = torch.randn(T, 1, generator=g, device=DEV)
    gr = 1e-2 * torch.randn(T, 1, generator=g, device=DEV)
    _, off, src, _ = gtr.permute(ids)
    gw, gx = gtr.route_backward(x, W, ids, z, gr, src, off, renormalize=False)
    s = torch.sigmoid(z.double())[:, 0]
    dz = s * (1 - s) * gr.double()[:, 0]
    dz_err = (32 + 8 * float(z.abs().max())) * U * dz.abs()
    at = torch.tensor([0, 1, 65_537, T // 2, (1 << 24) - 1, 1 << 24, T - 1], device=DEV)
    ref = dz[at, None] * W[ids[at, 0].long()].double()
    size = (dz_err[at] + 2 * U * dz[at].abs())[:, None] * W[ids[at, 0].long()].double().abs()
    within(gx[at], ref.cpu().numpy(),
           (1.01 * (size + u_of(BF) * (ref.abs() + size))).cpu().numpy(), "grad_x")
    want = torch.zeros(256, H, dtype=torch.float64, device=DEV)
    dz_part, sums = torch.zeros_like(want), torch.zeros_like(want)
    for t in range(0, T, 1 << 20):
        e, part = ids[t:t + (1 << 20), 0].long(), x[t:t + (1 << 20)].double()
        want.index_add_(0, e, dz[t:t + (1 << 20), None] * part)
        sums.index_add_(0, e, dz[t:t + (1 << 20), None].abs() * part.abs())
        dz_part.index_add_(0, e, dz_err[t:t + (1 << 20), None] * part.abs())
    chunks = int((off[1:] - off[:-1]).max()) // 256 + 1
    within(gw, want.cpu().numpy(),
           (1.01 * (dz_part + (40 + chunks) * U * sums)).cpu().numpy(), "grad_w_router")


@pytest.mark.parametrize("T", [60, 700])
def test_route_backward_a_dropped_pair_adds_nothing(T):
    # a sorted pair outside the batch has no token, so no token's infinities
    # reach the gradient through it
    say(f"[route_backward] a pair outside the batch beside an infinite row, T={T}")
    x, W, ids, z, g, src, off, _ = _router_case(T, 512, 8, T, 0.0, 6)
    others = torch.ones(256, dtype=torch.bool, device=DEV)
    others[ids[0].long()] = False  # the experts that token 0 did not choose
    at = int(others[ids.view(-1)[src.long()].long()].nonzero()[0])
    src[at] = -1
    want, _ = gtr.route_backward(x, W, ids, z, g, src, off)
    x[0] = float("inf")
    got, _ = gtr.route_backward(x, W, ids, z, g, src, off)
    assert torch.equal(got[others], want[others])
    assert bool(torch.isfinite(want).all()) and not bool(torch.isfinite(got[~others]).any())


def _route_reference(x, W, ids, z, g, renormalize, chunks, add=None):
    """(grad W, its bound, grad x, its bound) in fp64 on the device."""
    x, W, idn = x.double(), W.double(), ids.cpu().numpy()
    on = (idn >= 0) & (idn < 256)
    zz, gg = np.where(on, n64(z), 0.0), np.where(on, n64(g), 0.0)
    dz = train.route_dz(zz, idn, gg, renormalize)
    s = 1 / (1 + np.exp(-zz))
    if renormalize:
        w = np.where(on, s, 0.0)
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        size = w * (1 - s) * (np.abs(gg) + (np.abs(gg) * w).sum(1, keepdims=True))
    else:
        size = s * (1 - s) * np.abs(gg)
    err = (32 + 8 * np.abs(zz).max()) * U * size
    dev = lambda a: torch.from_numpy(a).to(DEV)
    dz, err = dev(dz), dev(np.where(on, err, 0.0))
    gw, bw = torch.zeros_like(W), torch.zeros_like(W)
    gx, bx = torch.zeros_like(x), torch.zeros_like(x)
    if add is not None:
        gx, bx = add.double(), 2 * U * add.double().abs()
    for j in range(ids.shape[1]):
        t = dev(np.nonzero(on[:, j])[0])
        e = ids[t, j].long()
        d, de = dz[t, j, None], err[t, j, None]
        gw.index_add_(0, e, d * x[t])
        bw.index_add_(0, e, (de + (40 + chunks) * U * d.abs()) * x[t].abs())
        gx[t] += d * W[e]
        bx[t] += (de + 20 * U * d.abs()) * W[e].abs()
    bx = bx + u_of(BF) * 1.01 * (gx.abs() + bx)
    return gw, 1.01 * bw, gx, 1.01 * bx


def _inside(got, ref, bound, what):
    """within() on the device."""
    worst = float(((got.double() - ref).abs() / bound.clamp(min=1e-300)).max())
    say(f"  {what}: largest error {worst:.3f} of its bound")
    assert worst <= 1, what


#: shares of 684, 429, 250 and 3200 tokens per workgroup of the kernel that
#: holds the weights in LDS, which takes 128 at a time: whole and partial last
#: turns, the ends of waves' tokens among them
@pytest.mark.parametrize("T,H,k,dropped", [(4099, 5120, 8, 0.02), (6001, 2304, 8, 0.0),
                                           (16000, 512, 3, 0.05), (6400, 16640, 2, 0.0)])
def test_route_backward_over_many_turns(T, H, k, dropped):
    say(f"[route_backward] T={T} H={H} k={k} dropped={dropped}")
    x, W, ids, z, g, src, off, add = _router_case(T, H, k, T, dropped, 8)
    chunks = int((off[1:] - off[:-1]).max()) // 256 + 1
    for extra in (None, add):
        gw, gx = gtr.route_backward(x, W, ids, z, g, src, off, grad_x_add=extra)
        rw, bw, rx, bx = _route_reference(x, W, ids, z, g, True, chunks, extra)
        _inside(gw, rw, bw, "grad_w_router")
        _inside(gx, rx, bx, "grad_x" if extra is None else "grad_x with add")
    # in place: the C call takes grad_x_add == grad_x
    cfg = gtr.make_config(T, H, 128, num_groups=1, topk_groups=1, topk=k)
    nb = gtr.workspace_bytes(cfg, gtr.ENTRY_ROUTE_BACKWARD)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    gw2, both = torch.empty_like(W), add.clone()
    st = gtr.lib().moe_route_backward(
        ctypes.byref(cfg), *(t.data_ptr() for t in (x, W, ids, z, g, src, off, both)), 0,
        gw2.data_ptr(), both.data_ptr(), ws.data_ptr(), nb,
        torch.cuda.current_stream(DEV).cuda_stream)
    assert st == 0
    assert torch.equal(gw2, gw) and torch.equal(both, gx)


@pytest.mark.parametrize("T,H,k,dt,dropped", [(7000, 5120, 8, BF, 0.02), (4500, 4099, 8, F, 0.0),
                                              (300_000, 136, 7, BF, 0.05)])
def test_rows_past_the_cached_size(T, H, k, dt, dropped):
    """Sorted rows of more than 512 MiB, which are stored past the caches: wide,
    odd and narrow rows, every call that writes them."""
    say(f"[rows] {T} x {k} x {H} {dt}: more than 512 MiB")
    assert T * k * H * dt.itemsize > 512 << 20
    g = torch.Generator(device=DEV).manual_seed(T)
    ids = torch.randint(0, 256, (T, k), generator=g, device=DEV, dtype=torch.int32)
    ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < dropped, -1, ids)
    _, off, _, dst = gtr.permute(ids)
    x = torch.randn(T, H, generator=g, device=DEV).to(dt)
    y = torch.randn(T * k, H, generator=g, device=DEV).to(dt)
    w = weights(T, k, 1)
    n = int(off[-1])
    d, on = dst.view(T, k).long(), dst.view(T, k) >= 0
    assert bool((on == (ids >= 0)).all()) and (dropped == 0) == (n == T * k)
    mark = torch.full((), 7.0, dtype=dt, device=DEV)

    def fresh():
        return mark.expand(T * k, H).contiguous()

    copied = gtr.dispatch(x, dst, topk=k, out=fresh())
    scaled = gtr.dispatch(x, dst, topk=k, topk_w=w, out=fresh())
    gy, gw = gtr.combine_backward(x, y, dst, w, out=fresh())
    gy_alone, none = gtr.combine_backward(x, None, dst, w, need_grad_w=False, out=fresh())
    assert none is None and torch.equal(gy_alone, gy)
    del gy_alone
    for got in (copied, scaled, gy):
        assert bool((got[n:] == 7).all())  # rows that no pair names
    u = u_of(dt)
    for j in range(k):
        t = on[:, j].nonzero()[:, 0]
        for a in range(0, len(t), 50_000):
            s = t[a:a + 50_000]
            r, xs, ws = d[s, j], x[s].double(), w[s, j, None].double()
            assert torch.equal(copied[r], x[s])
            for got, c, rounds in ((scaled, 1.0, 1), (gy, 2.5, 2)):
                ref = c * ws * xs
                assert bool(((got[r].double() - ref).abs()
                             <= (rounds * U + u) * 1.01 * ref.abs()).all())
            terms = xs * y[r].double()
            rounds = -(-H // 4096)
            assert bool(((gw[s, j].double() - 2.5 * terms.sum(1)).abs()
                         <= (24 + 8 * rounds) * U * 2.5 * terms.abs().sum(1)).all())
    assert float(gw[~on].abs().sum()) == 0


# ---------------------------------------------------------------------------
# RouterTrainer in the forms it can be built in
@pytest.mark.parametrize("kind", ["fp8", "packed", "sel_bias", "plain_weights", "groups",
                                  "scaling", "8bit"])
def test_router_trainer_forms(kind):
    """The output is the block's, the gradient that of the reference on the
    same expert outputs, the weights those of AdamW by itself on it."""
    say(f"[trainer] {kind}")
    T = 150
    d = synth.make_inputs(synth.workload("tiny", T=T), 0, device=DEV)
    x, W, gu, dn = d["x"], d["w_router"].clone(), d["w_gate_up"], d["w_down"]
    kw, layer, opt_kw, renormalize, scaling = {}, {}, {}, True, 2.5
    experts = (gu, dn)
    if kind == "fp8":
        experts = (gtr.quantize_fp8(gu, dn),)
    elif kind == "packed":
        experts = gtr.pack_weights(gu, dn)
        kw = layer = dict(weight_layout=gtr.LAYOUT_PACKED)
    elif kind == "sel_bias":
        kw = layer = dict(sel_bias=torch.linspace(-0.3, 0.3, 256, device=DEV))
    elif kind == "plain_weights":
        renormalize = False
        kw = layer = dict(renormalize=False)
    elif kind == "groups":
        kw = layer = dict(num_groups=1, topk_groups=1, topk=5)
    elif kind == "scaling":
        scaling = -0.75
        kw = layer = dict(routed_scaling=scaling)
    else:
        kw = opt_kw = dict(state_bits=8, seed=6)
    forward = gtr.layer_forward_fp8 if kind == "fp8" else gtr.layer_forward
    trainer = gtr.RouterTrainer(W, *experts, lr=1e-3, weight_decay=0.1, **kw)
    twin = W.clone()
    alone = gtr.AdamW([twin], lr=1e-3, weight_decay=0.1, **opt_kw)
    g = torch.Generator().manual_seed(1)
    for step in range(3):
        want = forward(x, W, *experts, **layer)
        out = trainer.forward(x)
        assert torch.equal(out, want)
        xs, ids, w, z, off, src, dst, y = trainer._saved
        go = (torch.randn(T, 256, generator=g) * 1e-2).to(BF).to(DEV)
        grad = n64(trainer.backward(go))
        idn, dn_ = ids.cpu().numpy(), dst.cpu().numpy()
        k = idn.shape[1]
        _, gw = train.combine_backward(n64(go), n64(y), dn_, n64(w), scaling)
        rw, _ = train.route_backward(n64(x), n64(W), idn, n64(z), gw, renormalize)
        size = abs(scaling) * train._dots(np.abs(n64(go)), np.abs(n64(y)), dn_, k) * (32 * U)
        dz_err = size + size.sum(1, keepdims=True)  # |w (1 - s)| and |s (1 - s)| are at most 1
        ew = np.zeros_like(rw)
        for j in range(k):
            np.add.at(ew, idn[:, j], dz_err[:, j, None] * np.abs(n64(x)))
        bw, _ = _route_bounds(n64(x), n64(W), idn, n64(z), gw, renormalize, T * k // 256 + 1)
        within(grad, rw, bw + ew, f"step {step} gradient")
        alone.step([trainer.grad])
        trainer.step()
        assert torch.equal(W, twin)


def test_adamw_names_what_is_not_aligned():
    say("[adamw] a gradient that starts inside 16 bytes")
    p = [torch.zeros(64, device=DEV), torch.zeros(32, device=DEV)]
    flat = torch.ones(97, device=DEV)
    for capturable in (False, True):
        opt = gtr.AdamW(p, capturable=capturable)
        with pytest.raises(gtr.MoeError, match=r"grads\[1\] is not 16-byte aligned"):
            opt.step([flat[:64], flat[65:]])
        assert opt.step_count == 0 and float(p[0].abs().max()) == 0
        with pytest.raises(gtr.MoeError, match="MOE_ERR_INVALID_ARG"):
            opt.step([flat[:64], None], lr=-1.0)
    with pytest.raises(gtr.MoeError, match=r"params\[0\] is not 16-byte aligned"):
        gtr.AdamW([flat[1:65]]).step([p[0]])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_c_call_takes_steps_of_list_and_tensors(bits):
    """In one call: a tensor with a step of its own, one with its own on the
    device, and one that goes by the list's, on the device or not."""
    say(f"[adamw] the C call's four places of a step, {bits} bits")
    sizes, own = (1000, 70, 2049), (3, 7, 12)
    counters = torch.tensor([7, 12], dtype=torch.int64, device=DEV)
    got = None
    for on_device in (False, True):
        params = [rows(1, n, F, i).view(-1) for i, n in enumerate(sizes)]
        grads = [rows(1, n, F, 10 + i).view(-1) for i, n in enumerate(sizes)]
        want = [p.clone() for p in params]
        ref = _opt(want, state_bits=bits, seed=3, step_count=[s - 1 for s in own])
        ref.step(grads)
        opt = _opt(params, state_bits=bits, seed=3)  # its states, and its list to fill in
        for d, g, n in zip(opt._list, grads, sizes):
            d.grad, d.grad_dtype, d.n = g.data_ptr(), gtr.DTYPE_FP32, n
        opt._list[0].step = 3
        opt._list[1].step, opt._list[1].step_dev = 99, counters.data_ptr()  # the device's goes first
        a = opt._opt
        a.lr, a.grad_scale, a.step = HP["lr"], 1.0, 1 if on_device else 12
        a.step_dev = counters.data_ptr() + 8 if on_device else None
        st = gtr.lib().moe_adamw_step(ctypes.byref(a), opt._list, 3,
                                      torch.cuda.current_stream(DEV).cuda_stream)
        assert st == 0
        for i in range(3):
            assert torch.equal(params[i], want[i]), (on_device, i)
            for k in ref.state:
                if ref.state[k][i] is not None:
                    assert torch.equal(opt.state[k][i].float(), ref.state[k][i].float()), (i, k)
        assert got is None or all(torch.equal(x, y) for x, y in zip(got, params))
        got = params
