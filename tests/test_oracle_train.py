"""Pins of the training calls' CPU reference: its gradients against autograd in
fp64 and against central differences, its 8-bit rounding against the format's
definition, its AdamW against the textbook recursion and torch's."""
import numpy as np
import pytest
import torch

import oracle
from oracle import train


def _case(T, H, k, E, seed, dropped=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int64)
    ids[rng.random((T, k)) < dropped] = -1
    counts, offsets, src, dst = oracle.permute(ids, E)
    return rng, ids, offsets, src, dst


def _index(dst, T, k):
    d = torch.from_numpy(np.asarray(dst).reshape(T, k).astype(np.int64))
    return d, d >= 0


@pytest.mark.parametrize("T,H,k,dropped", [(1, 5, 1, 0.0), (9, 7, 3, 0.0), (20, 6, 8, 0.2)])
def test_row_gradients_equal_autograd(T, H, k, dropped):
    rng, ids, _, _, dst = _case(T, H, k, 16, T, dropped)
    d, on = _index(dst, T, k)
    w = torch.from_numpy(rng.random((T, k))).requires_grad_()
    x = torch.from_numpy(rng.normal(size=(T, H))).requires_grad_()
    y = torch.from_numpy(rng.normal(size=(T * k, H))).requires_grad_()

    xp = torch.zeros(T * k, H, dtype=torch.float64).index_put(
        (d[on],), (w[:, :, None] * x[:, None, :])[on])
    assert np.allclose(train.dispatch(x.detach(), dst, k, w.detach()), xp.detach(), atol=1e-14)
    g = torch.from_numpy(rng.normal(size=(T * k, H)))
    gx, gw = torch.autograd.grad(xp, (x, w), g)
    rx, rw = train.dispatch_backward(g, dst, k, x.detach(), w.detach())
    assert np.allclose(rx, gx, atol=1e-13) and np.allclose(rw, gw, atol=1e-13)

    rows = torch.where(on[:, :, None], y[d.clamp(min=0)], 0.0)
    out = 2.5 * (w[:, :, None] * rows).sum(1)
    assert np.allclose(train.combine(y.detach(), dst, w.detach(), 2.5), out.detach(), atol=1e-13)
    go = torch.from_numpy(rng.normal(size=(T, H)))
    gy, gw = torch.autograd.grad(out, (y, w), go)
    ry, rw = train.combine_backward(go, y.detach(), dst, w.detach(), 2.5)
    assert np.allclose(ry, gy, atol=1e-13) and np.allclose(rw, gw, atol=1e-13)


def test_rows_that_no_pair_names_stay():
    _, _, _, _, dst = _case(6, 4, 3, 8, 1, 0.5)
    out = np.full((18, 4), 7.0)
    got = train.dispatch(np.ones((6, 4)), dst, 3, out=out)
    named = np.zeros(18, bool)
    named[dst[dst >= 0]] = True
    assert 0 < named.sum() < 18
    assert np.all(got[named] == 1.0) and np.all(got[~named] == 7.0)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_equals_autograd_and_differences(renormalize):
    T, H, k, E = 7, 10, 4, 12
    rng, ids, _, _, _ = _case(T, H, k, E, 3, 0.15)
    x0, W0, g = rng.normal(size=(T, H)), rng.normal(size=(E, H)), rng.normal(size=(T, k))
    on = torch.from_numpy(ids >= 0)
    idx = torch.from_numpy(np.maximum(ids, 0))

    def loss(x, W):
        s = torch.where(on, torch.sigmoid((x[:, None, :] * W[idx]).sum(2)), 0.0)
        if renormalize:
            s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
        return (s * torch.from_numpy(g)).sum()

    x, W = torch.from_numpy(x0).requires_grad_(), torch.from_numpy(W0).requires_grad_()
    gx, gW = torch.autograd.grad(loss(x, W), (x, W))
    logits = np.einsum("th,tjh->tj", x0, W0[np.maximum(ids, 0)])
    rW, rx = train.route_backward(x0, W0, ids, logits, g, renormalize)
    assert np.allclose(rW, gW, atol=1e-12) and np.allclose(rx, gx, atol=1e-12)
    add = rng.normal(size=(T, H))
    assert np.allclose(train.route_backward(x0, W0, ids, logits, g, renormalize, add)[1],
                       rx + add, atol=1e-14)
    # along one direction, by central differences
    dx, dW, h = rng.normal(size=(T, H)), rng.normal(size=(E, H)), 1e-5
    at = lambda s: float(loss(torch.from_numpy(x0 + s * dx), torch.from_numpy(W0 + s * dW)))
    slope = (at(h) - at(-h)) / (2 * h)
    assert abs(slope - ((rx * dx).sum() + (rW * dW).sum())) < 1e-7 * max(1.0, abs(slope))


def test_route_gradient_at_extreme_logits():
    g = np.array([[1.0, -2.0]])
    ids = np.array([[3, 9]])
    # saturated scores: the gradient vanishes, nothing is lost to 1 - s = 0
    dz = train.route_dz(np.array([[40.0, 41.0]]), ids, g, True)
    assert np.allclose(dz, [[0.5 * np.exp(-40) * 1.5, -0.5 * np.exp(-41) * 1.5]], rtol=1e-9)
    # scores that underflow keep their ratio
    dz = train.route_dz(np.array([[-900.0, -900.0]]), ids, g, True)
    assert np.allclose(dz, [[0.75, -0.75]], rtol=1e-12)
    assert np.all(train.route_dz(np.array([[-np.inf, -np.inf]]), ids, g, True) == 0)
    assert np.all(train.route_dz(np.zeros((1, 2)), np.array([[-1, 256]]), g, True) == 0)


def test_adamw_equals_torch_over_steps():
    rng = np.random.default_rng(0)
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1)
    p = rng.normal(size=50)
    t = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    m = v = np.zeros(50)
    for step in range(1, 8):
        g = rng.normal(size=50)
        t.grad = torch.from_numpy(g)
        opt.step()
        p, m, v = train.adamw(p, g, m, v, step=step, **hp)
    assert np.allclose(p, t.detach(), rtol=1e-12, atol=1e-13)


def test_block_scales_are_the_least_that_fit():
    for x, e in ((448.0, 0), (np.nextafter(448.0, 500), 1), (1.75, -8), (1.7500001, -7),
                 (1e-30, -108), (0.0, -126), (2.0 ** -130, -126), (3e38, 120), (np.inf, -126)):
        assert int(train.block_scales(np.array([x]))[0]) - 127 == e, x
    assert list(train.block_scales(np.r_[np.full(32, 448.0), 1.75])) == [127, 119]


def test_8bit_rounding_brackets_the_value_and_keeps_its_mean():
    rng = np.random.default_rng(5)
    x = np.r_[rng.normal(size=63) * 10.0 ** rng.uniform(-5, 2, 63), 0.0]
    total = np.zeros(64)
    draws = 4096
    for i in range(draws):
        # an even grid of the 16 random bits
        random = np.full(64, (i * 16) % 65536)
        code, scale = train.encode_8bit(x, random, False)
        got = train.decode_8bit(code, scale)
        step = _step(x, scale)
        assert np.all(np.abs(got - x) < step)
        total += got
    # the grid's spacing is 2^-12 of a step: the mean is off by at most that
    assert np.all(np.abs(total / draws - x) <= _step(x, scale) * (2.0 ** -12 + 1e-6))


def _step(x, scale):
    s = 2.0 ** (np.repeat(scale.astype(np.float64), 32)[:len(x)] - 127)
    a = np.maximum(np.abs(x) / s, 2.0 ** -6)
    return s * 2.0 ** (np.floor(np.log2(a)) - 3)


def test_8bit_special_values():
    x = np.r_[np.nan, np.inf, -1.0, 1e-9, np.zeros(28)]
    code, scale = train.encode_8bit(x, np.zeros(32, np.int64), True)
    assert code[0] & 0x7F == 0x7F and code[1] == 0x7F
    assert code[2] == 0xF8 and int(scale[0]) == 127 - 8  # 1 = 256 * 2^-8
    assert code[3] == 1 and np.all(code[4:] == 0)
    assert train.encode_8bit(x, np.zeros(32, np.int64), False)[0][3] == 0


def test_rounding_bits_are_spread():
    n = 1 << 16
    r = train.rounding_bits(7, 3, 2, n)
    for b in range(32):  # each bit is set in half of the elements, within 6 sigma
        assert abs(int(((r >> np.uint64(b)) & np.uint64(1)).sum()) - n / 2) < 6 * np.sqrt(n) / 2
    lo, hi = (r & np.uint64(0xFFFF)).astype(float), (r >> np.uint64(16)).astype(float)
    for a, b in ((lo, hi), (lo[1:], lo[:-1]), (hi[1:], hi[:-1])):
        assert abs(np.corrcoef(a, b)[0, 1]) < 6 / np.sqrt(n)
    for other in ((8, 3, 2), (7, 4, 2), (7, 3, 3)):
        o = (train.rounding_bits(*other, n) & np.uint64(0xFFFF)).astype(float)
        assert abs(np.corrcoef(lo, o)[0, 1]) < 6 / np.sqrt(n)


def test_stochastic_rounding_lets_a_small_change_through():
    # v decaying by 0.1 % a step: rounded to nearest its code would never move
    x = np.full(32, 288.0)  # a code's value
    nearest = train.encode_8bit(x * 0.9995, np.full(32, 32768), True)
    assert np.all(train.decode_8bit(*nearest) == 288.0)
    code, scale = train.encode_8bit(x, np.zeros(32, np.int64), True)
    start = train.decode_8bit(code, scale).mean()
    assert start == 288.0
    for step in range(1, 401):
        value = train.decode_8bit(code, scale) * 0.9995
        code, scale = train.encode_8bit(
            value, (train.rounding_bits(1, step, 0, 32) >> np.uint64(16)).astype(np.int64), True)
    # mean exp(-0.2) = 0.82 of the start; the walk's deviation per element is
    # below 0.3 of it, of the mean of 32 below 0.054
    assert abs(train.decode_8bit(code, scale).mean() / start - 0.9995 ** 400) < 6 * 0.054
