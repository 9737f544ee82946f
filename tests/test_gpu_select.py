"""Routing from logits on the GPU against the plain reference in fp64
(oracle/scores.py): selection, its gradient, the balance loss.

Ids are equal: values are compared in 64 bits on both sides, and the inputs'
neighbours are equal (ties, by index) or further apart than 2^-45 of their size.

Weights and gradients count roundings, U = u(fp32) = 2^-24:

* exp(d), d a difference of two fp32 numbers: d carries U |d|, the exponential
  2U, so U (2 + |d|) of its value; a sum of up to 1024 such terms at most 16 in a
  lane and 6 across: 22 U, plus its terms' mean U (2 + |d|).  A softmax score has
  both, a quotient or reciprocal and product (2U): with D = max |d| over the row,
  (28 + 2 D) U relative, which also holds for the sum's mean |d| <= D.  Terms
  below 2^-126 flush to zero in their own lane: 2^-126 absolute.
* a sigmoid: exp (2U + none: d = -z exactly), one addition, one quotient: 4U.
* a renormalised weight: the logarithm of the score (its size |l|: 4 U (1 +
  |l|) for the sigmoid's log1p, nothing for the softmax's logits), a difference
  and exponential as above, a sum of k, a quotient: with L the largest |l| of the
  chosen and D their spread, (40 + 8 L + 2 D) U.
* gradients are sums of products of these: relative to the sum of the
  magnitudes of the terms, twice the weights' bound (g w and its sum) plus 16 U
  for the products and additions; then u(bf16) |ref| where that is the type.
* the balance loss adds positive terms (a workgroup's tokens in fp32, at most
  per = ceil(T / 256) rounded up to 16 of them, then 64 bits): relative (per + 32)
  U plus a score's bound plus, for the sigmoid's sum over all experts, 22 U.
"""
import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
from oracle import scores as ref
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U, TINY = 2.0 ** -24, 2.0 ** -120
BF, F = torch.bfloat16, torch.float32


def n64(t):
    return t.detach().cpu().double().numpy()


def logits(T, E, dt, seed, masked=0.0, scale=1.5, empty=()):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * scale
    if masked:
        z[torch.rand(T, E, generator=g) < masked] = -float("inf")
    for t in empty:
        if t < T:
            z[t] = -float("inf")
    return z.to(dt).to(DEV)


def within(got, want, bound, what):
    got = n64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    err = np.where(np.isnan(want), 0.0, np.abs(got - want))  # NaN: on both sides
    bound = np.where(np.isnan(want), 0.0, bound)
    worst = float(np.max(err / np.maximum(bound, 1e-300), initial=0.0))
    say(f"  {what}: largest error {worst:.3f} of its bound")
    assert (err <= bound).all(), f"{what}: {worst:.3f} of its bound"


def spread(z):
    """max |z_e - max z| over a row's unmasked experts (and 0), capped where the
    score is below 2^-150 anyway."""
    z = np.nan_to_num(n64(z), nan=0.0, posinf=ref.F32_MAX)
    top = z.max(1, keepdims=True)
    d = np.where(z > -np.inf, top - z, 0.0)
    return np.minimum(d.max(1, keepdims=True), 104.0)


def weight_bound(z, ids, want, score, renormalize):
    """Relative bound of the weights, [T, 1]."""
    D = spread(z)
    if not renormalize:
        return (28 + 2 * D) * U if score == "softmax" else np.full_like(D, 5 * U)
    l = np.take_along_axis(ref.log_scores(n64(z), score), np.maximum(ids, 0), 1)
    l = np.where((ids >= 0) & (l > -np.inf), l, np.nan)
    with np.errstate(all="ignore"):
        big = np.nan_to_num(np.nanmax(np.abs(l), 1, keepdims=True, initial=0.0))
        wide = np.nan_to_num(np.nanmax(l, 1, keepdims=True, initial=-1e300, where=~np.isnan(l))
                             - np.nanmin(l, 1, keepdims=True, initial=1e300, where=~np.isnan(l)))
    return (40 + 8 * np.minimum(big, 1e4) + 2 * np.clip(wide, 0, 104)) * U


def check_select(z, what, **kw):
    got_ids, got_w = gtr.select(z, **{k: v for k, v in kw.items() if k != "bias"},
                                sel_bias=kw.get("bias"))
    args = {k: v for k, v in kw.items() if k != "bias"}
    bias = kw.get("bias")
    want_ids, want_w = ref.select(n64(z), sel_bias=None if bias is None else n64(bias), **args)
    assert np.array_equal(got_ids.cpu().numpy(), want_ids), what
    rel = weight_bound(z, want_ids, want_w, kw.get("score", "softmax"), kw.get("renormalize", True))
    within(got_w, want_w, rel * np.nan_to_num(want_w) + TINY, what)
    return got_ids, got_w


#: tokens, experts, groups, kept, best, slots: one token and one expert; counts
#: at and around 64, 128, 256, 512, 1024; groups of one expert; all slots
SELECT_CASES = [(1, 1, 1, 1, 2, 1), (1, 256, 8, 4, 2, 8), (3, 2, 2, 1, 2, 1), (5, 7, 1, 1, 1, 7),
                (9, 60, 3, 2, 1, 5), (17, 63, 7, 3, 2, 4), (33, 64, 64, 9, 2, 9), (2, 65, 5, 4, 2, 8),
                (31, 127, 1, 1, 2, 8), (70, 128, 16, 5, 1, 6), (12, 129, 3, 2, 2, 8),
                (130, 255, 5, 2, 2, 8), (257, 256, 1, 1, 2, 8), (64, 256, 64, 20, 2, 32),
                (19, 257, 1, 1, 2, 32), (40, 384, 6, 3, 2, 6), (23, 512, 8, 3, 2, 8),
                (11, 513, 27, 5, 1, 8), (8, 1000, 10, 4, 2, 16), (6, 1024, 32, 8, 2, 32),
                (1000, 16, 4, 2, 2, 2), (4, 33, 3, 3, 2, 32)]


@pytest.mark.parametrize("T,E,G,kg,best,k", SELECT_CASES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [F, BF], ids=["fp32", "bf16"])
def test_select(T, E, G, kg, best, k, score, dt):
    say(f"[select] T={T} E={E} G={G} kept={kg} best={best} k={k} {score} {dt}")
    kw = dict(score=score, num_groups=G, topk_groups=kg, group_best=best, topk=k)
    g = torch.Generator().manual_seed(E)
    bias = (torch.randn(E, generator=g) * (0.3 if score == "sigmoid" else 1.0 / E)).to(DEV)
    for i, (masked, renormalize, b) in enumerate([(0.0, True, None), (0.3, False, bias),
                                                  (0.0, False, None), (0.3, True, bias)]):
        z = logits(T, E, dt, 10 * T + i, masked, empty=(0, 5) if masked else ())
        check_select(z, f"masked={masked} renormalize={renormalize} bias={b is not None}",
                     renormalize=renormalize, bias=b, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(60, 5), (256, 8), (700, 16)])
def test_select_special_values(score, E, k):
    """Infinities, NaN, logits far out, rows without an expert, disabled experts."""
    say(f"[select] special values {score} E={E}")
    z = logits(24, E, F, 3)
    inf, nan = float("inf"), float("nan")
    z[0] = -inf
    z[1, 3:] = -inf                      # fewer experts than slots
    z[2, 7] = inf
    z[3, [2, 9]] = inf
    z[4, 5] = nan
    z[5] = nan
    z[6] = 3.0                           # all equal: the lowest indices
    z[7] = -200.0 - torch.arange(E, device=DEV)   # scores below fp32's range
    z[8] = 200.0 + torch.arange(E, device=DEV) * 0.5  # sigmoids of one
    z[9] = -3.4028234e38
    z[10, 0] = 3.4028234e38
    z[11] *= 1e-20
    z[12] = torch.where(torch.arange(E, device=DEV) % 2 == 0, 90.0, -90.0)
    z[13, :] = 0.0
    z[13, 4] = -0.0
    groups = dict(num_groups=4, topk_groups=2) if E % 4 == 0 else {}
    for renormalize in (True, False):
        check_select(z, f"renormalize={renormalize}", score=score, topk=k, renormalize=renormalize)
        check_select(z, "groups", score=score, topk=k, renormalize=renormalize, **groups)
    bias = torch.zeros(E, device=DEV)
    bias[[1, 2]], bias[3], bias[5] = -inf, nan, 0.25
    check_select(z, "bias", score=score, topk=k, bias=bias)
    check_select(z, "bias, groups", score=score, topk=k, bias=bias, **groups)
    bias[:] = -inf
    ids, w = gtr.select(z, score=score, topk=k, sel_bias=bias)
    assert (ids == -1).all() and (w[4:6].isnan().all() and (w[:4] == 0).all() and (w[6:] == 0).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_orders_values_closer_than_an_fp32_rounding(score):
    """Experts whose biased scores, and groups whose sums, differ by 2^-30."""
    say(f"[select] close values {score}")
    E, T = 64, 50
    z = torch.zeros(T, E, device=DEV)  # every score 1/2 or 1/64
    g = torch.Generator().manual_seed(0)
    steps = torch.randperm(E, generator=g).float()
    # exactly representable beside each other, not in a sum of 24 bits with 1/2
    bias = (steps * 2.0 ** -30).to(DEV)
    ids, _ = check_select(z, "bias", score=score, topk=8, bias=bias)
    assert ids[0].tolist() == torch.argsort(-steps)[:8].tolist()
    check_select(z, "groups", score=score, topk=8, bias=bias, num_groups=16, topk_groups=3)
    # logits one fp32 step apart
    z = (1.0 + torch.rand(T, E, generator=g).mul_(64).floor() * 2.0 ** -23).to(DEV)
    check_select(z, "logits", score=score, topk=8)
    check_select(z, "logits, groups", score=score, topk=8, num_groups=16, topk_groups=5)


def test_select_of_unaligned_rows():
    """Slices of a batch whose rows are not 16-byte aligned."""
    say("[select] unaligned")
    for dt, E in ((F, 257), (F, 256), (BF, 60), (BF, 129), (F, 6)):
        buf = logits(40, E, dt, 1).view(-1)
        for off in (1, 2, 3, 5):
            z = buf[off:off + 37 * E].view(37, E)
            ids, w = check_select(z, f"{dt} E={E} offset {off}", topk=4)
            want = gtr.select(z.clone(), topk=4)
            assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
            g = torch.randn(37, 4, device=DEV)
            loss, load = gtr.balance_loss(z, ids)
            assert torch.equal(loss, gtr.balance_loss(z.clone(), ids)[0])
            assert torch.equal(gtr.select_backward(z, ids, g, load=load),
                               gtr.select_backward(z.clone(), ids, g, load=load))


# ---------------------------------------------------------------------------
def random_ids(T, E, k, seed, dropped=0.0, padded=0.0, repeats=False):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    if repeats and k > 1:
        ids[::2, 1] = ids[::2, 0]
    ids[rng.random((T, k)) < dropped] = -1
    ids[rng.random((T, k)) < dropped / 2] = E + 3
    ids[rng.random(T) < padded] = -1
    return ids


def check_backward(z, ids, g, what, score, renormalize, load=None, gl=None):
    got = gtr.select_backward(z, torch.from_numpy(ids).to(DEV),
                              None if g is None else torch.from_numpy(g).to(DEV), score=score,
                              renormalize=renormalize, load=load, grad_loss=gl)
    assert got.dtype == z.dtype and got.shape == z.shape
    want, size = ref.select_backward(n64(z), ids, g, score=score, renormalize=renormalize,
                                     load=None if load is None else n64(load),
                                     grad_loss=1.0 if gl is None else float(gl))
    rel = np.zeros((z.shape[0], 1))
    if g is not None:
        rel = weight_bound(z, np.where((ids >= 0) & (ids < z.shape[1]), ids, -1), None, score,
                           renormalize)
    if load is not None:
        rel = np.maximum(rel, (60 + 2 * spread(z)) * U)
    u = torch.finfo(z.dtype).eps / 2
    bound = (2 * rel + 16 * U) * size + u * np.nan_to_num(np.abs(want))
    within(got, want, bound + TINY, what)
    return got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (17, 60, 4), (33, 63, 5),
                                   (9, 64, 8), (50, 65, 8), (31, 128, 6), (130, 255, 8),
                                   (300, 256, 8), (21, 257, 32), (13, 512, 8), (6, 1000, 16),
                                   (5, 1024, 32), (700, 16, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [F, BF], ids=["fp32", "bf16"])
def test_select_backward(T, E, k, score, dt):
    say(f"[select_backward] T={T} E={E} k={k} {score} {dt}")
    rng = np.random.default_rng(T + E)
    g = rng.normal(size=(T, k)).astype(np.float32)
    load = torch.from_numpy((rng.random(E) * 1e-2).astype(np.float32)).to(DEV)
    gl = torch.full((1,), 0.37, device=DEV)
    for renormalize in (True, False):
        z = logits(T, E, dt, T + 1)
        ids = random_ids(T, E, k, 5, 0.1, 0.2, repeats=True)
        check_backward(z, ids, g, "weights", score, renormalize)
        check_backward(z, ids, g, "weights and loss", score, renormalize, load, gl)
        check_backward(z, ids, None, "loss", score, renormalize, load)
        z = logits(T, E, dt, T + 2, 0.3, empty=(0,))
        check_backward(z, ids, g, "masked", score, renormalize, load, gl)
    none = np.full((T, k), -1, np.int32)
    out = check_backward(z, none, g, "no expert", score, True, load, gl)
    assert not out.any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_select_backward_special_values(score, renormalize):
    say(f"[select_backward] special values {score} renormalize={renormalize}")
    E, k = 60, 4
    z = logits(10, E, F, 1)
    z[0, 4] = float("nan")
    z[1, 4] = float("inf")
    z[2] = -200.0 - torch.arange(E, device=DEV)
    z[3] = 200.0
    z[4, 1:] = -float("inf")
    z[5, 3] = 60.0   # a score of one but for its last bits
    ids = random_ids(10, E, k, 2)
    ids[4] = [0, -1, 7, -1]  # an expert that the logits mask
    ids[5, 0] = 3
    ids[5, 1:] = [1, 2, 4]
    g = np.random.default_rng(0).normal(size=(10, k)).astype(np.float32)
    load = torch.rand(E, device=DEV) * 0.01
    check_backward(z, ids, g, "weights", score, renormalize)
    check_backward(z, ids, g, "weights and loss", score, renormalize, load)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_select_backward_equals_differences(score, renormalize):
    """Along random directions, against the call's own weights in fp64 (the
    reference's): third derivatives leave h^2, the gradient's bound U of its size."""
    say(f"[select_backward] differences {score} renormalize={renormalize}")
    z = logits(20, 48, F, 7)
    ids, _ = gtr.select(z, score=score, topk=6, renormalize=renormalize)
    at = ids.cpu().numpy()
    rng = np.random.default_rng(1)
    g = rng.normal(size=at.shape).astype(np.float32)
    grad = n64(gtr.select_backward(z, ids, torch.from_numpy(g).to(DEV), score=score,
                                   renormalize=renormalize))

    def value(x):
        s = np.take_along_axis(ref.scores(x, score), at, 1)
        return (g * (s / s.sum(1, keepdims=True) if renormalize else s)).sum()

    h = 1e-4
    for _ in range(4):
        d = rng.normal(size=z.shape)
        slope = (value(n64(z) + h * d) - value(n64(z) - h * d)) / (2 * h)
        assert abs(slope - (grad * d).sum()) <= 1e-5 * np.abs(grad * d).sum()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (15, 60, 4), (16, 64, 8),
                                   (17, 65, 8), (333, 160, 6), (1000, 256, 8), (4097, 128, 8),
                                   (20, 1000, 16), (700, 1024, 32), (9000, 8, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [F, BF], ids=["fp32", "bf16"])
def test_balance_loss(T, E, k, score, dt):
    say(f"[balance_loss] T={T} E={E} k={k} {score} {dt}")
    for masked, dropped, padded in ((0.0, 0.0, 0.0), (0.3, 0.1, 0.3)):
        z = logits(T, E, dt, T, masked, empty=(0,) if masked else ())
        ids = random_ids(T, E, k, 3, dropped, padded)
        loss, load = gtr.balance_loss(z, torch.from_numpy(ids).to(DEV), score=score, coef=0.03)
        assert loss.shape == () and load.shape == (E,)
        want, want_load = ref.balance_loss(n64(z), ids, score=score, coef=0.03)
        within(load, want_load, 4 * U * want_load, "load")
        per = -(-(-(-T // 256)) // 16) * 16
        rel = (per + 32 + 22 + 28 + 2 * spread(z).max()) * U
        within(n64(loss).reshape(1), np.array([want]), np.array([rel * want + TINY]), "loss")


def test_balance_loss_without_rows_and_with_nan():
    say("[balance_loss] no rows, NaN")
    z = logits(30, 64, F, 1)
    none = torch.full((30, 4), -1, dtype=torch.int32, device=DEV)
    loss, load = gtr.balance_loss(z, none)
    assert float(loss) == 0 and not load.any()
    z[7, 3] = float("nan")
    loss, load = gtr.balance_loss(z, none)
    assert float(loss) == 0 and not load.any()  # the row is not one of the loss's
    none[7, 0] = 5
    loss, load = gtr.balance_loss(z, none)
    assert loss.isnan() and load.isfinite().all()


def test_training_step_of_a_softmax_router():
    """The calls together, as a training step makes them around the block's own:
    route_select, permute, experts in 4 bits, combine and back."""
    say("[chain] route_select to router gradient")
    T, H, I, k, coef = 150, 512, 256, 6, 0.02
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    W = (torch.randn(256, H, generator=g) * 0.05).to(DEV)
    w4 = gtr.quantize_fp4((torch.randn(256, 2 * I, H, generator=g) * 0.02).to(BF).to(DEV),
                          (torch.randn(256, H, I, generator=g) * 0.02).to(BF).to(DEV))
    ids, w, z = gtr.route_select(x, W, topk=k, return_logits=True)
    again = gtr.select(z, topk=k)
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)
    assert torch.equal(gtr.route_select(x, W, topk=k)[0], ids)
    exact = n64(x) @ n64(W).T
    within(z, exact, (H + 32) * U * (np.abs(n64(x)) @ np.abs(n64(W)).T), "logits")
    counts, off, src, dst = gtr.permute(ids)
    y = gtr.expert_ffn_fp4(x, src, off, w4, topk=k)
    out = gtr.combine(y, dst, w)
    loss, load = gtr.balance_loss(z, ids, coef=coef)
    assert int(counts.sum()) == T * k and out.isfinite().all()
    go = (torch.randn(T, H, generator=g) * 1e-2).to(BF).to(DEV)
    _, gw = gtr.combine_backward(go, y, dst, w, need_grad_y=False)
    gz = gtr.select_backward(z, ids, gw, load=load)
    want, size = ref.select_backward(n64(z), ids.cpu().numpy(), n64(gw), load=n64(load))
    within(gz, want, (2 * (60 + 2 * spread(z)) + 16) * U * size + U * np.abs(want), "grad logits")

    def total(zz):  # the step's loss by the logits, routing and experts fixed
        p = ref.scores(zz, "softmax")
        c = np.take_along_axis(p, ids.cpu().numpy(), 1)
        return ((c / c.sum(1, keepdims=True)) * n64(gw)).sum() + (n64(load) * p).sum()

    d, h = np.random.default_rng(3).normal(size=want.shape), 1e-4
    slope = (total(n64(z) + h * d) - total(n64(z) - h * d)) / (2 * h)
    assert abs(slope - (n64(gz) * d).sum()) <= 1e-5 * np.abs(n64(gz) * d).sum()


def test_captured_calls_replay():
    """Two graphs of the whole set, on two streams at once, replayed with eager
    work and new inputs between: every replay gives the eager bits."""
    say("[graph] two graphs, replayed")

    def chain(z, g):
        ids, w = gtr.select(z, topk=4, num_groups=4, topk_groups=2)
        loss, load = gtr.balance_loss(z, ids)
        return ids, w, loss, load, gtr.select_backward(z, ids, g, load=load, grad_loss=loss)

    ins = [(logits(500 + 77 * i, 64, F, i), torch.randn(500 + 77 * i, 4, device=DEV))
           for i in range(2)]
    graphs, outs = [], []
    for z, g in ins:
        chain(z, g)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(chain(z, g))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for z, _ in ins:
            z.copy_(logits(*z.shape, F, 10 + i))
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for (z, g), got in zip(ins, outs):
            for a, b in zip(got, chain(z, g)):
                assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_side_streams_and_repeated_calls_give_the_same_bits():
    say("[streams] two at once, and again")
    z, ids = logits(3000, 256, F, 2), None
    want = None
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = torch.randn(3000, 8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                ids, w = gtr.select(z)
                loss, load = gtr.balance_loss(z, ids)
                got.append((ids, w, loss, load, gtr.select_backward(z, ids, g, load=load)))
        torch.cuda.synchronize()
        want = want or got[0]
        for r in got:
            assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_a_workspace_of_the_callers():
    say("[balance_loss] workspace")
    ws = gtr.Workspace()
    for T in (10, 5000, 300):
        z = logits(T, 256, F, T)
        ids, _ = gtr.select(z)
        a, b = gtr.balance_loss(z, ids, workspace=ws), gtr.balance_loss(z, ids)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_empty_batches():
    say("[empty] no tokens")
    z = torch.zeros(0, 64, device=DEV)
    ids, w = gtr.select(z, topk=4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    loss, load = gtr.balance_loss(z, ids)
    assert float(loss) == 0 and load.shape == (64,) and not load.any()
    torch.set_default_dtype(torch.float64)
    try:
        loss, load = gtr.balance_loss(z, ids)
    finally:
        torch.set_default_dtype(torch.float32)
    assert loss.dtype == load.dtype == torch.float32
    assert gtr.select_backward(z, ids, w).shape == (0, 64)
    ids, w, zz = gtr.route_select(torch.zeros(0, 256, dtype=BF, device=DEV),
                                  torch.zeros(256, 256, device=DEV), return_logits=True)
    assert ids.shape == (0, 8) and zz.shape == (0, 256)


def test_large_batches():
    """More elements than 31 bits count: the last rows as a small batch's."""
    say("[select] 2^31 elements and more")
    T, E, k = (1 << 21) + 3, 1024, 2
    z = torch.zeros(T, E, dtype=BF, device=DEV)
    last = logits(300, E, BF, 1)
    z[-300:] = last
    ids, w = gtr.select(z, topk=k)
    a = gtr.select(last, topk=k)
    assert torch.equal(ids[-300:], a[0]) and torch.equal(w[-300:], a[1])
    assert (ids[:1000] == torch.tensor([0, 1], device=DEV)).all()
    g = torch.randn(T, k, device=DEV)
    gz = gtr.select_backward(z, ids, g)
    assert torch.equal(gz[-300:], gtr.select_backward(last, a[0], g[-300:].contiguous()))
    ids[:-300] = -1
    loss, load = gtr.balance_loss(z, ids)
    want, _ = ref.balance_loss(n64(last), a[0].cpu().numpy())
    assert abs(float(loss) - want) <= ((T // 256 + 200) * U) * want
