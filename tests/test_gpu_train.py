"""The training calls on the GPU against the plain reference in fp64.

Tolerances count roundings.  u(t) = torch.finfo(t).eps / 2 is the largest
relative error of one rounding to t; with U = u(fp32) = 2^-24:

* a copy is exact; a weighted row is one fp32 product and one rounding:
  (U + u(t)) |ref|, with one more product for the combine's scale;
* a sum over k slots has at most k products and k additions: 2k U times the sum
  of the terms' magnitudes (plus the scale's product), then u(t) |ref|;
* a dot product over a row is at most 8 terms in a thread and column round (H up
  to 8192 bf16 or 4096 fp32 is one round), 6 additions across a wave, 15 across
  waves and the scale: 32 U times the sum of the magnitudes (a row of up to 32
  pieces: 8 terms and 5 additions);
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
             (2, 33000, 3, 0.0), (6, 40, 8, 1.0),
             (37, 9, 8, 0.1), (1000, 64, 8, 0.05), (77, 129, 8, 0.0), (50, 130, 7, 0.1)]


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
               (31, 768, 8, 0.0, 0), (32, 256, 8, 0.0, 0), (33, 256, 8, 0.05, 0), (128, 2304, 8, 0.05, 4), (129, 2304, 8, 0.05, 4),
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


@pytest.mark.parametrize("T", [60, 700])
def test_route_backward_drops_what_lies_outside(T):
    """Offsets outside the rows are cut to them, sorted pairs outside the batch
    are left out (the kernels check both, so nothing outside is touched)."""
    say(f"[route_backward] perm_src and offsets outside the batch, T={T}")
    x, W, ids, z, g, src, off, _ = _router_case(T, 512, 8, T, 0.0, 6)
    n = T * 8
    want = gtr.route_backward(x, W, ids, z, g, src, off)
    cut = off.clone()
    cut[0], cut[256] = -7, n + 5000
    for a, b in zip(gtr.route_backward(x, W, ids, z, g, src, cut), want):
        assert torch.equal(a, b)
    bad = src.clone()
    at = [0, 5, n // 2, n - 1]
    bad[at] = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    gw, gx = gtr.route_backward(x, W, ids, z, g, bad, off)
    assert torch.equal(gx, want[1])
    idn, dz = ids.cpu().numpy(), train.route_dz(n64(z), ids.cpu().numpy(), n64(g), True)
    ref = train.route_backward(n64(x), n64(W), idn, n64(z), n64(g))[0]
    for p in src.cpu().numpy()[at]:
        ref[idn[p // 8, p % 8]] -= dz[p // 8, p % 8] * n64(x)[p // 8]
    bw, _ = _route_bounds(n64(x), n64(W), idn, n64(z), n64(g), True, n // 256 + 1)
    within(gw, ref, bw, "grad_w_router")
    # offsets that run backwards give experts no rows
    back = torch.flip(off, [0]).contiguous()
    assert float(gtr.route_backward(x, W, ids, z, g, src, back)[0].abs().max()) == 0


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


def test_adamw_zero_gradients_from_a_zero_state():
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
    with pytest.raises(ValueError, match="listed twice"):
        _opt([p, p])
    with pytest.raises(ValueError, match="contiguous"):
        _opt([torch.zeros(8, 8, device=DEV).t()])
    with pytest.raises(gtr.MoeError):  # a view that is not 16-byte aligned
        o = _opt([p[1:]])
        o.step([torch.zeros(63, device=DEV)])
    with pytest.raises(gtr.MoeError):
        _opt([p]).step([torch.zeros(64, device=DEV)], lr=-1.0)
    with pytest.raises(ValueError, match="one element"):
        _opt([p]).step([torch.zeros(64, device=DEV)], lr=torch.zeros(2, device=DEV))
    moved = torch.zeros(64, device=DEV)
    o = _opt([moved])
    moved.data = torch.ones(128, device=DEV)
    with pytest.raises(RuntimeError, match="lies elsewhere"):
        o.step([torch.zeros(64, device=DEV)])
    with pytest.raises(ValueError, match="state must hold"):
        _opt([p], state={"exp_avg": [p]})
    assert float(p.abs().max()) == 0


# ---------------------------------------------------------------------------
# together, as they are used
def _tiny(T, seed=0):
    w = synth.workload("tiny", T=T)
    d = synth.make_inputs(w, seed, device=DEV)
    return d["x"], d["w_router"], d["w_gate_up"], d["w_down"]


@pytest.mark.parametrize("T,replay", [(40, False), (300, False), (300, True)])
def test_router_training_steps(T, replay):
    """Three steps of RouterTrainer: the output is the block's bit for bit, the
    gradient that of the staged reference on the same expert outputs, and the
    weights those of AdamW on that gradient."""
    say(f"[trainer] T={T} replay={replay}")
    x, W, gu, dn = _tiny(T)
    W = W.clone()
    ids_in = None
    if replay:
        ids_in = gtr.route(x, W)[0].clone()
        ids_in[2, 3], ids_in[5] = -1, 400
    trainer = gtr.RouterTrainer(W, gu, dn, lr=1e-3, weight_decay=0.1)
    g = torch.Generator().manual_seed(1)
    p, m, v = n64(W), 0.0 * n64(W), 0.0 * n64(W)
    for step in (1, 2, 3):
        if not replay:
            want = gtr.layer_forward(x, W, gu, dn)
        for micro in range(2):  # two micro-batches accumulate
            go = (torch.randn(T, 256, generator=g) * 1e-2).to(BF).to(DEV)
            out = trainer.forward(x, ids_in)
            if not replay:
                assert torch.equal(out, want)
            xs, ids, w, z, off, src, dst, y = trainer._saved
            before = None if trainer.grad is None else n64(trainer.grad)
            grad = n64(trainer.backward(go))
            idn, d = ids.cpu().numpy(), dst.cpu().numpy()
            _, gw = train.combine_backward(n64(go), n64(y), d, n64(w), 2.5)
            rw, _ = train.route_backward(n64(x), n64(W), idn, n64(z), gw)
            # the weights' gradient carries 32 U of its terms' magnitudes
            size = 2.5 * train._dots(np.abs(n64(go)), np.abs(n64(y)), d, 8) * (32 * U)
            on = (idn >= 0) & (idn < 256)
            dz_err = np.where(on, size + size.sum(1, keepdims=True), 0.0)  # |w (1 - s)| <= 1
            ew = np.zeros_like(rw)
            for j in range(8):
                t = np.nonzero(on[:, j])[0]
                np.add.at(ew, idn[t, j], dz_err[t, j, None] * np.abs(n64(x))[t])
            bw, _ = _route_bounds(n64(x), n64(W), idn, n64(z), gw, True, T * 8 // 256 + 1)
            if before is not None:
                rw, bw = rw + before, bw + U * (np.abs(rw) + np.abs(before))
            within(grad, rw, bw + ew, f"step {step} gradient {micro}")
        total = n64(trainer.grad)
        start = n64(W)
        trainer.step(grad_scale=0.5)
        assert trainer.grad is None
        m0, v0 = m, v
        _, m, v = train.adamw(start, total, m0, v0, step=step, lr=1e-3, beta1=0.9, beta2=0.999,
                              eps=1e-8, weight_decay=0.1, grad_scale=0.5)
        ref = train.adamw(start, total, m0, v0, step=step, lr=1e-3, beta1=0.9, beta2=0.999,
                          eps=1e-8, weight_decay=0.1, grad_scale=0.5)[0]
        # an update is at most lr / (1 - beta1) here; its error a few hundred U
        # of that (m and v carry up to `step` roundings each)
        within(W, ref, 4 * U * np.abs(start) + 1e-2 * 256 * U, f"step {step} weights")
        m, v = n64(trainer.optimizer.state["exp_avg"][0]), n64(trainer.optimizer.state["exp_avg_sq"][0])
    with pytest.raises(RuntimeError, match="no gradient"):
        trainer.step()
    with pytest.raises(RuntimeError, match="no forward"):
        trainer.backward(go)


def test_router_gradient_equals_differences():
    """The chain combine -> router against central differences of the block in
    fp64, routing and expert outputs fixed."""
    say("[trainer] differences")
    T = 64
    x, W, gu, dn = _tiny(T, 3)
    trainer = gtr.RouterTrainer(W.clone(), gu, dn)
    trainer.forward(x)
    _, ids, _, _, _, _, dst, y = trainer._saved
    go = (torch.randn(T, 256, generator=torch.Generator().manual_seed(2)) * 1e-2).to(BF).to(DEV)
    grad = n64(trainer.backward(go))
    X, Y, G, idn = n64(x), n64(y), n64(go), ids.cpu().numpy().astype(np.int64)
    dots = train._dots(G, Y, dst.cpu().numpy(), 8)

    def loss(w64):
        s = 1 / (1 + np.exp(-np.take_along_axis(X @ w64.T, idn, 1)))
        return 2.5 * float(((s / s.sum(1, keepdims=True)) * dots).sum())

    rng, w0 = np.random.default_rng(0), n64(W)
    for _ in range(4):
        d = rng.normal(size=w0.shape)
        h = 1e-4
        slope = (loss(w0 + h * d) - loss(w0 - h * d)) / (2 * h)
        # the gradient's fp32 error along d, from its entries' scale; third
        # derivatives leave h^2 of it
        assert abs(slope - (grad * d).sum()) <= 1e-4 * np.abs(grad * d).sum(), slope


@pytest.mark.parametrize("dt,H", [(F, 100), (BF, 256)], ids=["fp32", "bf16"])
def test_own_experts_between_dispatch_and_combine(dt, H):
    """A caller's trainable experts (each scales its rows by a vector): the
    gradients of x, the weights and the experts against the reference."""
    say(f"[own experts] {dt} H={H}")
    T, k = 90, 4
    ids, off, src, dst = routing(T, k, 8, 0.1)
    d = dst.cpu().numpy()
    x, w, a = rows(T, H, dt, 1), weights(T, k, 2), rows(256, H, F, 3)
    n = int(off[-1])
    e_of = torch.repeat_interleave(torch.arange(256, device=DEV), off[1:].long() - off[:-1].long())
    xp = gtr.dispatch(x, dst, topk=k, out=torch.zeros(T * k, H, dtype=dt, device=DEV))
    y = torch.zeros_like(xp)
    y[:n] = (xp[:n].float() * a[e_of]).to(dt)
    out = gtr.combine(y, dst, w, routed_scaling=2.5)
    _sum_close(out, n64(y), d, n64(w), 2.5, dt, "out")
    go = rows(T, H, dt, 4)
    gy, gw = gtr.combine_backward(go, y, dst, w, out=torch.zeros_like(y))
    grad_a = torch.zeros(256, H, device=DEV).index_add_(0, e_of, gy[:n].float() * xp[:n].float())
    gxp = torch.zeros_like(gy)
    gxp[:n] = (gy[:n].float() * a[e_of]).to(dt)
    gx = gtr.dispatch_backward(gxp, dst, topk=k)
    # the reference from the definition, per token and slot
    X, A, Wt, G = n64(x), n64(a), n64(w), n64(go)
    rx, rA, rw = np.zeros((T, H)), np.zeros((256, H)), np.zeros((T, k))
    size_x, size_w, size_A = np.zeros((T, H)), np.zeros((T, k)), np.zeros((256, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            rx[t] += 2.5 * Wt[t, j] * G[t] * A[e]
            size_x[t] += np.abs(2.5 * Wt[t, j] * G[t] * A[e])
            rA[e] += 2.5 * Wt[t, j] * G[t] * X[t]
            size_A[e] += np.abs(2.5 * Wt[t, j] * G[t] * X[t])
            rw[t, j] = 2.5 * (G[t] * X[t] * A[e]).sum()
            size_w[t, j] = 2.5 * np.abs(G[t] * X[t] * A[e]).sum()
    # roundings to dt on the way: gy and gxp (x), gy (A), y (w), then sums
    u = u_of(dt)
    within(gx, rx, (3.1 * u + 24 * U) * size_x, "grad x")
    within(grad_a, rA, (1.1 * u + 64 * U) * size_A, "grad experts")
    within(gw, rw, (1.1 * u + 40 * U) * size_w, "grad weights")


def test_captured_training_step_replays():
    """Forward, backward and a capturable AdamW step in one graph, replayed with
    eager work and new inputs between: every replay gives the eager bits."""
    say("[graph] a captured step, replayed five times")
    T = 200
    x, W0, gu, dn = _tiny(T, 5)
    lr = torch.full((1,), 1e-3, device=DEV)
    scale = torch.full((1,), 1.0, device=DEV)

    def chain(xx, go, W, opt):
        ids, w, z = gtr.route(xx, W, return_logits=True)
        _, off, src, dst = gtr.permute(ids)
        y = gtr.expert_ffn(xx, src, off, gu, dn)
        out = gtr.combine(y, dst, w)
        gy, gw = gtr.combine_backward(go, y, dst, w)
        xp = gtr.dispatch(xx, dst)
        gx = gtr.dispatch_backward(gy, dst)
        gW, gx = gtr.route_backward(xx, W, ids, z, gw, src, off, grad_x_add=gx)
        opt.step([gW], lr=lr, grad_scale=scale)
        return out, gx, gW, xp

    for bits in (32, 8):
        Wc, We = W0.clone(), W0.clone()
        oc = gtr.AdamW([Wc], state_bits=bits, seed=9, capturable=True)
        oe = gtr.AdamW([We], state_bits=bits, seed=9)
        xs, gos = x.clone(), torch.zeros(T, 256, dtype=BF, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # warm up, then undo
            chain(xs, gos, Wc, oc)
        torch.cuda.current_stream().wait_stream(side)
        Wc.copy_(W0)
        for name in oc.state:
            for t in oc.state[name]:
                if t is not None:
                    t.view(torch.uint8).zero_()
        oc._step_dev.zero_()
        assert oc.step_count == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(xs, gos, Wc, oc)
        g = torch.Generator().manual_seed(4)
        for i in range(5):
            xs.copy_(torch.randn(T, 256, generator=g).to(BF))
            gos.copy_((torch.randn(T, 256, generator=g) * 1e-2).to(BF))
            lr.fill_(1e-3 / (i + 1))
            scale.fill_(1.0 + 0.25 * i)
            graph.replay()
            torch.cuda.synchronize()
            want = chain(xs, gos, We, oe)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b), (bits, i)
            assert torch.equal(Wc, We), (bits, i)
            for name in oc.state:
                for a, b in zip(oc.state[name], oe.state[name]):
                    assert a is None or torch.equal(a.float(), b.float()), (bits, i, name)
        assert oc.step_count == oe.step_count == 5


def test_two_captured_graphs_do_not_share_scratch():
    say("[graph] two graphs of the router's gradient on two streams at once")
    cases = [_router_case(1500, 768, 8, s, 0.0, 8) for s in (1, 2)]
    want = [gtr.route_backward(*c[:7], grad_x_add=c[7]) for c in cases]
    graphs, got = [], []
    for c in cases:
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(gtr.route_backward(*c[:7], grad_x_add=c[7]))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for gw, gx in got:
            gw.zero_(), gx.zero_()
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for (gw, gx), (rw, rx) in zip(got, want):
            assert torch.equal(gw, rw) and torch.equal(gx, rx)


def test_side_streams_and_repeated_calls_give_the_same_bits():
    say("[streams] calls on two side streams at once, and again")
    x, W, ids, z, g, src, off, add = _router_case(900, 1280, 8, 3)
    dst = torch.empty_like(src)
    dst[src.long()] = torch.arange(900 * 8, device=DEV, dtype=torch.int32)
    w, y = weights(900, 8, 1), rows(900 * 8, 1280, BF, 2)

    def all_of():
        return (*gtr.route_backward(x, W, ids, z, g, src, off, grad_x_add=add),
                gtr.dispatch(x, dst, topk_w=w), *gtr.dispatch_backward(y, dst, x=x, topk_w=w),
                *gtr.combine_backward(x, y, dst, w))

    want = all_of()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(all_of())
        torch.cuda.synchronize()
        for r in got:
            for a, b in zip(r, want):
                assert torch.equal(a, b)


def test_capture_needs_a_capturable_optimizer():
    say("[graph] AdamW without capturable=True")
    p, g = torch.zeros(64, device=DEV), torch.ones(64, device=DEV)
    opt = gtr.AdamW([p])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="capturable"):
            opt.step([g])
    assert opt.step_count == 0


def test_empty_batches_and_lists():
    say("[empty] no tokens")
    i = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    z = lambda *s, dt=F: torch.zeros(*s, dtype=dt, device=DEV)
    assert gtr.dispatch(z(0, 7), i(0)).shape == (0, 7)
    assert gtr.dispatch_backward(z(0, 7), i(0)).shape == (0, 7)
    gy, gw = gtr.combine_backward(z(0, 7), z(0, 7), i(0), z(0, 8))
    assert gy.shape == (0, 7) and gw.shape == (0, 8)
    assert gtr.combine(z(0, 7), i(0), z(0, 8)).shape == (0, 7)
    W = rows(256, 256, F, 1)
    args = (z(0, 256, dt=BF), W, i(0).view(0, 8), z(0, 8), z(0, 8), i(0), i(257))
    gW, gx = gtr.route_backward(*args)
    assert gx.shape == (0, 256) and float(gW.abs().max()) == 0
    acc = torch.ones_like(W)
    assert gtr.route_backward(*args, grad_w_router=acc)[0] is acc and float(acc.min()) == 1
