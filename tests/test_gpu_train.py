"""The training calls on the GPU against the plain reference in fp64.

Tolerances count roundings.  u(t) = torch.finfo(t).eps / 2 is the largest
relative error of one rounding to t; with U = u(fp32) = 2^-24:

* a copy is exact; a weighted row is one fp32 product and one rounding:
  (U + u(t)) |ref|, with one more product for the combine's scale;
* a sum over k slots has at most k products and k additions: 2k U times the sum
  of the terms' magnitudes (plus the scale's product), then u(t) |ref|;
* a dot product over a row is at most 8 terms in a thread and column round (H up
  to 8192 bf16 or 4096 fp32 is one round), 6 additions across a wave, 15 across
  waves and the scale: 32 U times the sum of the magnitudes;
* dz of the router goes through log-sigmoids, exponentials and a quotient.  The
  exponent's absolute error is at most U (4 + 4 max|z|) (log1p and its
  difference, the maximum's own, their difference) and turns into a relative
  one; each exponential (1 ulp = 2U), sum of k and quotient adds a few U:
  (32 + 8 max|z|) U times w (1 - s) (|g| + sum |g| w);
* the router weights' gradient adds at most 32 rows per lane of a chunk of 256,
  1 + 3 additions across lanes and waves, then one per chunk: (40 + chunks) U
  times the sum of the magnitudes on top of dz's error.
"""
import ctypes

import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
import oracle
import synth
from oracle import train
from parity_util import say, to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
NAMES = {BF: "bf16", F: "fp32"}


def u_of(dt):
    return torch.finfo(dt).eps / 2


def n64(t):
    return t.detach().cpu().double().numpy()


def within(got, ref, bound, what):
    got = n64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (got.shape, ref.shape)
    over = np.abs(got - ref) - bound
    worst = float(np.max(np.abs(got - ref) / np.maximum(bound, 1e-300))) if got.size else 0.0
    say(f"  {what}: largest error {worst:.3f} of its bound")
    assert np.all(over <= 0), f"{what}: error {worst:.3f} of its bound"


def routing(T, k, seed, dropped=0.0, E=256, hot=0):
    """ids int32 [T, k] and permute's outputs, from the reference."""
    rng = np.random.default_rng(seed)
    key = rng.random((T, E))
    if hot:
        key[:, :hot] += 0.9
    ids = np.argsort(-key, 1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < dropped] = -1
    _, offsets, src, dst = oracle.permute(ids, E)
    # the entries behind the last row name nothing and must not be read
    src = np.concatenate([src, np.full(T * k - len(src), 2 ** 30)])
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)
    return ids, dev(offsets), dev(src), dev(dst)


def rows(T, H, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(dt).to(DEV)


def weights(T, k, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, k, generator=g) * 0.3).to(DEV)


#: tokens, width, slots, dropped share: one token and one element; widths below,
#: at and past a wave's piece and a workgroup; odd widths; every slot count
ROW_CASES = [(1, 1, 1, 0.0), (1, 5120, 8, 0.0), (3, 7, 2, 0.4), (5, 8, 3, 0.0), (17, 63, 4, 0.1),
             (33, 257, 5, 0.0), (64, 512, 8, 0.0), (31, 777, 6, 0.2), (130, 1023, 7, 0.05),
             (9, 4097, 8, 0.1), (40, 5120, 8, 0.0), (4, 8200, 8, 0.0), (700, 256, 8, 0.0),
             (2, 33000, 3, 0.0), (6, 40, 8, 1.0)]


@pytest.mark.parametrize("T,H,k,dropped", ROW_CASES)
@pytest.mark.parametrize("dt", [BF, F], ids=NAMES.get)
def test_dispatch(T, H, k, dropped, dt):
    say(f"[dispatch] T={T} H={H} k={k} dropped={dropped} {dt}")
    _, _, _, dst = routing(T, k, T + H, dropped)
    x, w = rows(T, H, dt, 1), weights(T, k, 2)
    start = rows(T * k, H, dt, 3)
    d = to_np(dst.float()).astype(np.int64)
    got = gtr.dispatch(x, dst, topk=k, out=start.clone())
    assert np.array_equal(n64(got), train.dispatch(n64(x), d, k, out=n64(start)))
    got = gtr.dispatch(x, dst, topk=k, topk_w=w, out=start.clone())
    ref = train.dispatch(n64(x), d, k, n64(w), out=n64(start))
    named = np.zeros(T * k, bool)
    named[d[d >= 0]] = True
    assert np.array_equal(n64(got)[~named], n64(start)[~named])
    within(got, ref, (U + u_of(dt)) * 1.01 * np.abs(ref) * named[:, None], "weighted")


@pytest.mark.parametrize("T,H,k,dropped", ROW_CASES)
@pytest.mark.parametrize("dt", [BF, F], ids=NAMES.get)
def test_dispatch_backward(T, H, k, dropped, dt):
    say(f"[dispatch_backward] T={T} H={H} k={k} dropped={dropped} {dt}")
    _, _, _, dst = routing(T, k, T + H, dropped)
    x, w, g = rows(T, H, dt, 1), weights(T, k, 2), rows(T * k, H, dt, 3)
    d = to_np(dst.float()).astype(np.int64)
    _sum_close(gtr.dispatch_backward(g, dst, topk=k), n64(g), d, np.ones((T, k)), 1.0, dt, "sum")
    gx, gw = gtr.dispatch_backward(g, dst, topk=k, x=x, topk_w=w)
    _sum_close(gx, n64(g), d, n64(w), 1.0, dt, "weighted sum")
    _dot_close(gw, n64(x), n64(g), d, k, 1.0, "weights")
    assert torch.equal(gtr.dispatch_backward(g, dst, topk=k, topk_w=w), gx)


def _rounds(H, dt):
    return -(-H // (8192 if dt == BF else 4096))


def _sum_close(got, b, d, w, scale, dt, what):
    ref = train.combine(b, d, w, scale)
    size = train.combine(np.abs(b), d, np.abs(w), abs(scale))
    err = (2 * w.shape[1] + 2) * U * size
    within(got, ref, err + u_of(dt) * 1.01 * (np.abs(ref) + err), what)


def _dot_close(got, a, b, d, k, scale, what):
    H = a.shape[1]
    ref = scale * train._dots(a, b, d, k)
    size = abs(scale) * train._dots(np.abs(a), np.abs(b), d, k)
    within(got, ref, (24 + 8 * _rounds(H, F)) * U * size, what)


@pytest.mark.parametrize("T,H,k,dropped", ROW_CASES)
@pytest.mark.parametrize("dt", [BF, F], ids=NAMES.get)
def test_combine_rows_and_backward(T, H, k, dropped, dt):
    say(f"[combine] T={T} H={H} k={k} dropped={dropped} {dt}")
    _, _, _, dst = routing(T, k, T + H, dropped)
    y, w, g = rows(T * k, H, dt, 1), weights(T, k, 2), rows(T, H, dt, 3)
    d = to_np(dst.float()).astype(np.int64)
    _sum_close(gtr.combine(y, dst, w, routed_scaling=2.5), n64(y), d, n64(w), 2.5, dt, "combine")
    start = rows(T * k, H, dt, 4)
    gy, gw = gtr.combine_backward(g, y, dst, w, routed_scaling=2.5, out=start.clone())
    ref = train.dispatch(n64(g), d, k, 2.5 * n64(w), out=n64(start))
    named = np.zeros(T * k, bool)
    named[d[d >= 0]] = True
    assert np.array_equal(n64(gy)[~named], n64(start)[~named])
    within(gy, ref, (2 * U + u_of(dt)) * 1.01 * np.abs(ref) * named[:, None], "grad_y")
    _dot_close(gw, n64(g), n64(y), d, k, 2.5, "grad_w")
    # either gradient alone is the same
    only_y, none = gtr.combine_backward(g, None, dst, w, need_grad_w=False, out=start.clone())
    assert none is None and torch.equal(only_y, gy)
    none, only_w = gtr.combine_backward(g, y, dst, w, need_grad_y=False)
    assert none is None and torch.equal(only_w, gw)


def test_row_indices_outside_the_rows_are_dropped():
    say("[rows] perm_dst outside the rows")
    T, H, k = 12, 40, 4
    _, _, _, dst = routing(T, k, 5)
    bad = dst.clone()
    bad[3], bad[10], bad[20] = T * k, -7, 2 ** 31 - 1
    gone = dst.clone()
    gone[[3, 10, 20]] = -1
    for dt in (BF, F):
        x, g, w, z = rows(T, H, dt, 1), rows(T * k, H, dt, 2), weights(T, k, 3), \
            torch.zeros(T * k, H, dtype=dt, device=DEV)
        assert torch.equal(gtr.dispatch(x, bad, topk=k, topk_w=w, out=z.clone()),
                           gtr.dispatch(x, gone, topk=k, topk_w=w, out=z.clone()))
        for a, b in zip(gtr.dispatch_backward(g, bad, topk=k, x=x, topk_w=w),
                        gtr.dispatch_backward(g, gone, topk=k, x=x, topk_w=w)):
            assert torch.equal(a, b)
        for a, b in zip(gtr.combine_backward(x, g, bad, w, out=z.clone()),
                        gtr.combine_backward(x, g, gone, w, out=z.clone())):
            assert torch.equal(a, b)
        assert float(gtr.combine_backward(x, g, bad, w)[1].view(-1)[[3, 10, 20]].abs().max()) == 0


def test_rows_with_infinities_and_nan():
    say("[rows] infinities, NaN, and NaN behind dropped pairs")
    T, H, k = 4, 24, 2
    dst = torch.tensor([0, 1, 2, -1, 3, 4, 5, 6], dtype=torch.int32, device=DEV)
    for dt in (BF, F):
        g = rows(T * k, H, dt, 1)
        g[7] = float("nan")  # a row that no pair names
        g[3, 2], g[0, 1] = float("inf"), float("nan")
        w = torch.ones(T, k, device=DEV)
        out = n64(gtr.dispatch_backward(g, dst, topk=k, topk_w=w))
        assert np.isinf(out[2, 2]) and np.isnan(out[0, 1])
        out[2, 2] = out[0, 1] = 0
        assert np.all(np.isfinite(out))
        x = rows(T, H, dt, 2)
        _, gw = gtr.combine_backward(x, g, dst, w)
        gw = n64(gw).ravel()
        assert np.isnan(gw[0]) and not np.isfinite(gw[4]) and gw[3] == 0
        assert np.all(np.isfinite(gw[[1, 2, 3, 5, 6, 7]]))
        x[1, 5] = float("nan")
        got = gtr.dispatch(x, dst, topk=k, out=torch.zeros(T * k, H, dtype=dt, device=DEV))
        assert np.isnan(n64(got)[2, 5]) and np.isnan(n64(got)).sum() == 1


def test_rows_past_4_gb():
    # byte offsets past 2^32 in the sorted rows
    say("[rows] 420000 tokens of 640 fp32 elements, 8 slots: 8.6 GB")
    T, H, k = 420_000, 640, 8
    g = torch.Generator(device=DEV).manual_seed(0)
    ids = torch.randint(0, 256, (T, k), generator=g, device=DEV, dtype=torch.int32)
    _, _, _, dst = gtr.permute(ids)
    x = torch.randn(T, H, generator=g, device=DEV)
    xp = gtr.dispatch(x, dst, topk=k)
    at = torch.tensor([0, 1, 12345, T // 2, T - 2, T - 1], device=DEV)
    d = dst.view(T, k)[at].long()
    assert int(d.max()) * H * 4 > 2 ** 32
    for j in range(k):
        assert torch.equal(xp[d[:, j]], x[at])
    gx = gtr.dispatch_backward(xp, dst, topk=k)
    # 8 additions of sums up to 8 |x| (x may be 0)
    assert bool(((gx - 8 * x).abs() <= 8 * 9 * U * x.abs()).all())


# ---------------------------------------------------------------------------
# the router
def _route_bounds(x, W, ids, z, g, renormalize, chunks):
    """Error bounds of grad_w_router and of grad_x before its rounding."""
    on = (ids >= 0) & (ids < 256)
    zz = np.where(on, z, 0.0)
    s = 1 / (1 + np.exp(-zz))
    rest = 1 / (1 + np.exp(zz))
    gg = np.where(on, np.abs(g), 0.0)
    if renormalize:
        w = np.where(on, s, 0.0)
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        size = w * rest * (gg + (gg * w).sum(1, keepdims=True))
    else:
        size = s * rest * gg
    dz_err = (32 + 8 * np.abs(zz).max()) * U * size
    dz = np.abs(train.route_dz(z, ids, g, renormalize))
    ew, sw, ex, sx = np.zeros_like(W), np.zeros_like(W), np.zeros_like(x), np.zeros_like(x)
    for j in range(ids.shape[1]):
        t = np.nonzero(on[:, j])[0]
        e = ids[t, j]
        np.add.at(ew, e, dz_err[t, j, None] * np.abs(x[t]))
        np.add.at(sw, e, dz[t, j, None] * np.abs(x[t]))
        ex[t] += dz_err[t, j, None] * np.abs(W[e])
        sx[t] += dz[t, j, None] * np.abs(W[e])
    return 1.01 * (ew + (40 + chunks) * U * sw), 1.01 * (ex + 18 * U * sx)


def _router_case(T, H, k, seed, dropped=0.0, hot=0, spread=1.5):
    ids, off, src, _ = routing(T, k, seed, dropped, hot=hot)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    W = (0.02 * torch.randn(256, H, generator=g)).to(DEV)
    z = (spread * torch.randn(T, k, generator=g)).to(DEV)
    gw = (1e-2 * torch.randn(T, k, generator=g)).to(DEV)
    add = (1e-2 * torch.randn(T, H, generator=g)).to(BF).to(DEV)
    return x, W, torch.from_numpy(ids).to(DEV), z, gw, src, off, add


ROUTE_CASES = [(1, 256, 1, 0.0, 0), (1, 5120, 8, 0.0, 0), (5, 512, 3, 0.3, 0),
               (31, 768, 8, 0.0, 0), (32, 256, 8, 0.0, 0), (33, 256, 8, 0.05, 0),
               (100, 1280, 5, 0.0, 8), (700, 512, 8, 0.02, 8), (3000, 256, 8, 0.0, 12),
               (4096, 256, 8, 0.0, 0), (4099, 512, 3, 0.05, 8),
               (4, 256, 8, 1.0, 0)]


@pytest.mark.parametrize("T,H,k,dropped,hot", ROUTE_CASES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward(T, H, k, dropped, hot, renormalize):
    say(f"[route_backward] T={T} H={H} k={k} dropped={dropped} hot={hot} renorm={renormalize}")
    x, W, ids, z, g, src, off, add = _router_case(T, H, k, T + H, dropped, hot)
    args = (x, W, ids, z, g, src, off)
    gw, gx = gtr.route_backward(*args, renormalize=renormalize)
    idn = ids.cpu().numpy()
    ref_w, ref_x = train.route_backward(n64(x), n64(W), idn, n64(z), n64(g), renormalize)
    bw, bx = _route_bounds(n64(x), n64(W), idn, n64(z), n64(g), renormalize, T * k // 256 + 1)
    within(gw, ref_w, bw, "grad_w_router")
    within(gx, ref_x, bx + u_of(BF) * 1.01 * (np.abs(ref_x) + bx), "grad_x")
    # experts without a token get exact zeros
    seen = np.zeros(256, bool)
    seen[idn[idn >= 0]] = True
    assert np.all(n64(gw)[~seen] == 0)
    # added to what is there, and to the other part of grad_x
    acc = torch.randn(256, H, device=DEV)
    start = acc.clone()
    gw2, gx2 = gtr.route_backward(*args, renormalize=renormalize, grad_x_add=add,
                                  grad_w_router=acc)
    assert gw2 is acc
    assert torch.equal(gw2, start + gw)
    ref = ref_x + n64(add)
    b = bx + 2 * U * (np.abs(n64(add)) + np.abs(ref_x))
    within(gx2, ref, b + u_of(BF) * 1.01 * (np.abs(ref) + b), "grad_x with add")
    # in place, and without grad_x
    gw3, gx3 = gtr.route_backward(*args, renormalize=renormalize, grad_x_add=add)
    assert torch.equal(gx3, gx2) and torch.equal(gw3, gw)
    gw4, none = gtr.route_backward(*args, renormalize=renormalize, need_grad_x=False)
    assert none is None and torch.equal(gw4, gw)


def test_route_backward_repeated_and_foreign_ids():
    say("[route_backward] the same expert twice in a token, ids outside the experts")
    T, H, k = 40, 256, 4
    rng = np.random.default_rng(3)
    ids = rng.integers(0, 6, (T, k)).astype(np.int32)
    ids[5, 1], ids[9, 0], ids[11] = 256, -5, -1
    _, off, src, _ = oracle.permute(ids, 256)
    src = np.concatenate([src, np.full(T * k - len(src), -9)])
    x, W, _, z, g, _, _, _ = _router_case(T, H, k, 9)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)
    gw, gx = gtr.route_backward(x, W, t(ids), z, g, t(src), t(off))
    rw, rx = train.route_backward(n64(x), n64(W), ids, n64(z), n64(g))
    bw, bx = _route_bounds(n64(x), n64(W), ids, n64(z), n64(g), True, 2)
    within(gw, rw, bw, "grad_w_router")
    within(gx, rx, bx + u_of(BF) * 1.01 * (np.abs(rx) + bx), "grad_x")
    assert float(gx[11].abs().max()) == 0


@pytest.mark.parametrize("T", [37, 5000])
def test_route_backward_adds_in_place(T):
    # the C call allows grad_x_add to be grad_x itself
    say(f"[route_backward] in place, T={T}")
    x, W, ids, z, g, src, off, add = _router_case(T, 768, 8, T, 0.02)
    want_w, want_x = gtr.route_backward(x, W, ids, z, g, src, off, grad_x_add=add)
    cfg = gtr.make_config(T, 768, 128, num_groups=1, topk_groups=1)
    nb = gtr.workspace_bytes(cfg, gtr.ENTRY_ROUTE_BACKWARD)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    gw, gx = torch.empty_like(W), add.clone()
    st = gtr.lib().moe_route_backward(
        ctypes.byref(cfg), *(t.data_ptr() for t in (x, W, ids, z, g, src, off, gx)), 0,
        gw.data_ptr(), gx.data_ptr(), ws.data_ptr(), nb,
        torch.cuda.current_stream(DEV).cuda_stream)
    assert st == 0
    assert torch.equal(gw, want_w) and torch.equal(gx, want_x)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_at_extreme_logits(renormalize):
    say(f"[route_backward] logits of +-30 and +-90, infinities; renorm={renormalize}")
    T, H, k = 64, 256, 4
    x, W, ids, z, g, src, off, _ = _router_case(T, H, k, 21)
    z = z * 0 + torch.tensor([30.0, -30.0, 90.0, -90.0], device=DEV)[
        torch.randint(0, 4, (T, k), generator=torch.Generator().manual_seed(1)).to(DEV)]
    gw, gx = gtr.route_backward(x, W, ids, z, g, src, off, renormalize=renormalize)
    idn = ids.cpu().numpy()
    rw, rx = train.route_backward(n64(x), n64(W), idn, n64(z), n64(g), renormalize)
    bw, bx = _route_bounds(n64(x), n64(W), idn, n64(z), n64(g), renormalize, T * k // 256 + 1)
    within(gw, rw, bw + 1e-38, "grad_w_router")
    within(gx, rx, bx + u_of(BF) * 1.01 * (np.abs(rx) + bx) + 1e-38, "grad_x")
    z[:] = -float("inf")
    gw, gx = gtr.route_backward(x, W, ids, z, g, src, off, renormalize=renormalize)
    assert float(gw.abs().max()) == 0 and float(gx.abs().max()) == 0
    z[:] = float("inf")
    gw, gx = gtr.route_backward(x, W, ids, z, g, src, off, renormalize=renormalize)
    assert float(gw.abs().max()) == 0 and float(gx.abs().max()) == 0


def test_route_logits_are_the_chosen_experts():
    say("[route_logits]")
    d = synth.make_inputs("tiny", 0, device=DEV)
    x, W = d["x"], d["w_router"]
    bias = torch.linspace(-0.2, 0.2, 256, device=DEV)
    for kw in (dict(), dict(sel_bias=bias), dict(renormalize=False, topk=5), dict(num_groups=1, topk_groups=1)):
        ids, w = gtr.route(x, W, **kw)
        ids2, w2, z = gtr.route(x, W, return_logits=True, **kw)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
        exact = np.take_along_axis(n64(x) @ n64(W).T, ids.cpu().numpy().astype(np.int64), 1)
        size = np.take_along_axis(np.abs(n64(x)) @ np.abs(n64(W)).T,
                                  ids.cpu().numpy().astype(np.int64), 1)
        # fp32 accumulation of H = 256 terms, each in three exact parts
        within(z, exact, 3 * 256 * U * size, "logits")
        r = ids.clone()
        r[3, 1], r[7, 0] = -1, 300
        w1 = gtr.route_replay(x, W, r, renormalize=kw.get("renormalize", True))
        w2, z2 = gtr.route_replay(x, W, r, renormalize=kw.get("renormalize", True),
                                  return_logits=True)
        assert torch.equal(w1, w2)
        same = (r >= 0) & (r < 256)
        assert torch.equal(z2[same], z[same]) and float(z2[~same].abs().max()) == 0


# ---------------------------------------------------------------------------
# AdamW
HP = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.05)


def _opt(params, **kw):
    return gtr.AdamW(params, lr=HP["lr"], betas=(HP["beta1"], HP["beta2"]), eps=HP["eps"],
                     weight_decay=HP["weight_decay"], **kw)


def _adam_bounds(p, g, m, v, step, gs, got_m=None):
    """Error bounds of (p, m, v) of one fp32 step from fp32 inputs: every
    constant and operation is one rounding."""
    b1, b2, lr, eps = HP["beta1"], HP["beta2"], HP["lr"], HP["eps"]
    G = np.abs(g * gs)
    em = U * (4 * b1 * np.abs(m) + 5 * (1 - b1) * G)
    ev = U * (4 * b2 * v + 8 * (1 - b2) * G * G)
    _, m1, v1 = train.adamw(p, g, m, v, step=step, grad_scale=gs, **HP)
    root = np.sqrt(v1 / (1 - b2 ** step))
    den = root + eps
    # sqrt halves v's relative error; root, scale, sum, quotient, factor
    rel = np.where(v1 > 0, 0.5 * ev / np.maximum(v1, 1e-300), 0.0) + 10 * U
    upd = lr / (1 - b1 ** step) / den
    ep = 4 * U * np.abs(p) + upd * (1.01 * em + np.abs(m1) * rel)
    return 1.01 * ep, 1.01 * em, 1.01 * ev


SIZES = [(1,), (7,), (8,), (31,), (32,), (33,), (5, 401), (2048,), (2049,), (3, 0), (100_003,)]


@pytest.mark.parametrize("pdt", [F, BF], ids=NAMES.get)
@pytest.mark.parametrize("gdt", [F, BF], ids=NAMES.get)
def test_adamw_32(pdt, gdt):
    say(f"[adamw] 32-bit states, params {pdt}, grads {gdt}")
    params = [rows(1, int(np.prod(s)), pdt, i).view(s) for i, s in enumerate(SIZES)]
    opt = _opt(params)
    for step in (1, 2, 3):
        before = [(n64(opt.state["master"][i] if pdt == BF else p), n64(opt.state["exp_avg"][i]),
                   n64(opt.state["exp_avg_sq"][i])) for i, p in enumerate(params)]
        grads = [rows(1, p.numel(), gdt, 100 * step + i).view(p.shape) * 0.1
                 for i, p in enumerate(params)]
        opt.step(grads, grad_scale=0.25)
        for i, (p, g) in enumerate(zip(params, grads)):
            p0, m0, v0 = before[i]
            if p.numel() == 0:
                continue
            ref = train.adamw(p0, n64(g), m0, v0, step=step, grad_scale=0.25, **HP)
            bounds = _adam_bounds(p0, n64(g), m0, v0, step, 0.25)
            new = opt.state["master"][i] if pdt == BF else p
            for a, r, b, name in zip((new, opt.state["exp_avg"][i], opt.state["exp_avg_sq"][i]),
                                     ref, bounds, ("p", "m", "v")):
                within(a, r, b, f"step {step} tensor {i} {name}")
            if pdt == BF:
                assert torch.equal(p, new.to(BF))  # the master to nearest
    assert opt.step_count == 3


@pytest.mark.parametrize("pdt", [F, BF], ids=NAMES.get)
@pytest.mark.parametrize("gdt", [F, BF], ids=NAMES.get)
def test_adamw_8bit(pdt, gdt):
    say(f"[adamw] 8-bit states, params {pdt}, grads {gdt}")
    params = [rows(1, int(np.prod(s)), pdt, i).view(s) for i, s in enumerate(SIZES)]
    opt = _opt(params, state_bits=8, seed=77)
    st = opt.state
    for step in (1, 2, 3):
        dec = lambda k, i: train.decode_8bit(st[k][i].view(torch.uint8).cpu().numpy().ravel(),
                                             st[k + "_scale"][i].view(torch.uint8).cpu().numpy())
        before = [(n64(st["master"][i] if pdt == BF else p).ravel(), dec("exp_avg", i),
                   dec("exp_avg_sq", i)) for i, p in enumerate(params)]
        # magnitudes over many decades within a block
        grads = [(rows(1, p.numel(), F, 100 * step + i)
                  * 10 ** (2.5 * rows(1, p.numel(), F, 200 * step + i).clamp(-2, 1))).to(gdt).view(p.shape)
                 for i, p in enumerate(params)]
        opt.step(grads, grad_scale=0.5)
        for i, (p, g) in enumerate(zip(params, grads)):
            if p.numel() == 0:
                continue
            p0, m0, r0 = before[i]
            gn = n64(g).ravel()
            f32 = np.float32
            m, v, root = train.adamw_state_f32(gn, m0, f32(r0) * f32(r0), beta1=HP["beta1"],
                                               beta2=HP["beta2"], grad_scale=0.5)
            bits = train.rounding_bits(77, step, i, p.numel())
            for k, x, b, low in (("exp_avg", m, bits & np.uint64(0xFFFF), False),
                                 ("exp_avg_sq", root, bits >> np.uint64(16), True)):
                code, scale = train.encode_8bit(x, b, low)
                assert np.array_equal(st[k + "_scale"][i].view(torch.uint8).cpu().numpy(), scale)
                got = st[k][i].view(torch.uint8).cpu().numpy().ravel()
                assert np.array_equal(train.decode_8bit(got, scale),
                                      train.decode_8bit(code, scale)), (step, i, k)
            # the update goes by the states before their rounding
            v0 = r0 * r0
            ref = train.adamw(p0, gn, m0, v0, step=step, grad_scale=0.5, **HP)[0]
            new = (st["master"][i] if pdt == BF else p).view(-1)
            within(new, ref, _adam_bounds(p0, gn, m0, v0, step, 0.5)[0], f"step {step} tensor {i}")
            if pdt == BF:
                assert torch.equal(p.view(-1), new.to(BF))


def test_adamw_many_tensors_of_both_kinds():
    # more tensors than one launch takes, fp32 and bf16 mixed, some skipped
    say("[adamw] 131 tensors, mixed types, some without a gradient")
    rng = np.random.default_rng(0)
    sizes = [int(s) for s in rng.integers(1, 5000, 131)]
    for bits in (32, 8):
        params = [rows(1, n, BF if i % 3 else F, i).view(-1) for i, n in enumerate(sizes)]
        alone = [p.clone() for p in params]
        grads = [None if i % 10 == 4 else rows(1, n, BF if i % 2 else F, 500 + i).view(-1)
                 for i, n in enumerate(sizes)]
        opt = _opt(params, state_bits=bits, seed=5)
        opt.step(grads)
        opt.step(grads)
        for i, p in enumerate(alone):
            if grads[i] is None:
                assert torch.equal(p, params[i])
                assert float(opt.state["exp_avg"][i].float().abs().max()) == 0
                continue
            if bits == 8 and i:
                continue  # the rounding goes by the place in the list
            o = _opt([p], state_bits=bits, seed=5)
            o.step([grads[i]])
            o.step([grads[i]])
            assert torch.equal(p, params[i]), i
            assert torch.equal(o.state["exp_avg"][0].float(), opt.state["exp_avg"][i].float())


def test_adamw_gradients_that_are_not_finite_stay_alone():
    say("[adamw] NaN and infinite gradients")
    for bits in (32, 8):
        p = rows(1, 100, F, 1).view(-1)
        clean = p.clone()
        g = rows(1, 100, F, 2).view(-1)
        bad = g.clone()
        bad[5], bad[40], bad[99] = float("nan"), float("inf"), -float("inf")
        a, b = _opt([p], state_bits=bits, seed=1), _opt([clean], state_bits=bits, seed=1)
        a.step([bad])
        b.step([g])
        fine = torch.ones(100, dtype=torch.bool, device=DEV)
        fine[[5, 40, 99]] = False
        assert torch.equal(p[fine], clean[fine])
        assert not torch.isfinite(p[~fine]).any()
        # a later step keeps it to these elements too
        a.step([g])
        assert torch.isfinite(p[fine]).all() and not torch.isfinite(p[~fine]).any()
        m = a.state["exp_avg"][0].float()
        assert torch.isfinite(m[fine]).all() and not torch.isfinite(m[~fine]).any()


def test_adamw_zero_gradients_and_zero_eps():
    say("[adamw] zero gradients from a zero state")
    for bits in (32, 8):
        p = rows(1, 70, F, 1).view(-1)
        before = p.clone()
        _opt([p], state_bits=bits).step([torch.zeros(70, device=DEV)])
        # 0 / (0 + eps): weight decay alone
        keep = np.float32(1 - HP["lr"] * HP["weight_decay"])
        assert np.array_equal(p.cpu().numpy(), before.cpu().numpy() * keep)


def test_adamw_state_continues_from_a_checkpoint():
    say("[adamw] state= and step_count=")
    for bits in (32, 8):
        for dt in (F, BF):
            p = [rows(1, n, dt, n).view(-1) for n in (50, 3000)]
            g = [[rows(1, n, dt, n + s).view(-1) for n in (50, 3000)] for s in (1, 2, 3)]
            a = _opt(p, state_bits=bits, seed=3)
            a.step(g[0])
            a.step(g[1])
            q = [t.clone() for t in p]
            state = {k: [None if t is None else t.clone() for t in v] for k, v in a.state.items()}
            b = _opt(q, state_bits=bits, seed=3, state=state, step_count=a.step_count)
            a.step(g[2])
            b.step(g[2])
            for x, y in zip(p, q):
                assert torch.equal(x, y)
            for k in state:
                for x, y in zip(a.state[k], state[k]):
                    assert (x is None and y is None) or torch.equal(x.float(), y.float())


def test_adamw_refuses():
    p = torch.zeros(64, device=DEV)
    with pytest.raises(ValueError, match="gradients expected"):
        _opt([p]).step([])
    with pytest.raises(ValueError, match="shape"):
        _opt([p]).step([torch.zeros(63, device=DEV)])
    with pytest.raises(TypeError):
        _opt([p]).step([torch.zeros(64, dtype=torch.float16, device=DEV)])
    with pytest.raises(ValueError, match="contiguous"):
        _opt([torch.zeros(8, 8, device=DEV).t()])
    with pytest.raises(gtr.MoeError):  # a view that is not 16-byte aligned
        o = _opt([p[1:]])
        o.step([torch.zeros(63, device=DEV)])
    with pytest.raises(gtr.MoeError):
        _opt([p]).step([torch.zeros(64, device=DEV)], lr=-1.0)
    with pytest.raises(ValueError, match="one element"):
        _opt([p]).step([torch.zeros(64, device=DEV)], lr=torch.zeros(2, device=DEV))
    with pytest.raises(ValueError, match="state must hold"):
        _opt([p], state={"exp_avg": [p]})
    assert float(p.abs().max()) == 0
