"""The reference of routing from logits and of the 4-bit weights (oracle/scores.py,
oracle/fp4.py) against hand cases, torch autograd in fp64, differences and the
formats' definitions."""
import numpy as np
import pytest
import torch

from oracle import fp4
from oracle import scores as ref


def _z(T, E, seed, scale=1.5):
    return np.random.default_rng(seed).normal(size=(T, E)) * scale


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_hand_case(score):
    z = np.array([[0.0, 2.0, 1.0, 2.0, -np.inf, 3.0]])
    ids, w = ref.select(z, score=score, topk=4, renormalize=False)
    assert ids.tolist() == [[5, 1, 3, 2]]  # the tie goes to the lower index
    s = 1 / (1 + np.exp(-z[0])) if score == "sigmoid" else np.exp(z[0]) / np.exp(z[0]).sum()
    np.testing.assert_allclose(w[0], s[[5, 1, 3, 2]], rtol=1e-14)
    # two groups of three: 0 + 2 + 1 against 2 + (masked) + 3
    ids, w = ref.select(z, score=score, num_groups=2, topk_groups=1, group_best=2, topk=3)
    assert ids.tolist() == [[5, 3, -1]] and w[0, 2] == 0
    np.testing.assert_allclose(w.sum(), 1.0, rtol=1e-14)
    # a bias moves the choice, not the weights
    bias = np.array([9.0, 0, 0, 0, 9.0, -np.inf])
    ids, w = ref.select(z, score=score, sel_bias=bias, topk=2, renormalize=False)
    assert ids.tolist() == [[0, 1]]
    np.testing.assert_allclose(w[0], s[[0, 1]], rtol=1e-14)


def test_select_empty_and_nan_rows():
    z = np.full((3, 4), -np.inf)
    z[1, 2], z[2, 1], z[2, 0] = 1.0, np.nan, 0.5
    ids, w = ref.select(z, topk=2)
    assert ids.tolist() == [[-1, -1], [2, -1], [0, -1]]
    assert w[0].tolist() == [0, 0] and w[1].tolist() == [1, 0] and np.isnan(w[2]).all()
    ids, w = ref.select(np.array([[np.inf, 0.0, np.inf]]), topk=2)
    assert ids.tolist() == [[0, 2]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("load", [True, False])
def test_gradient_is_autograds(score, renormalize, load):
    T, E, k, coef = 7, 20, 4, 0.05
    z = _z(T, E, 1)
    z[2, 5] = -np.inf
    ids, _ = ref.select(z, score=score, topk=k)
    ids[3, 1], ids[4] = -1, -1  # a dropped slot, a padded row
    ids[5, 2] = ids[5, 0]       # the same expert twice
    g = np.random.default_rng(2).normal(size=(T, k))
    zt = torch.tensor(z, requires_grad=True)
    s = torch.sigmoid(zt) if score == "sigmoid" else torch.softmax(zt, 1)
    on = torch.tensor(ids >= 0)
    w = torch.where(on, s.gather(1, torch.tensor(ids).clamp(min=0).long()), 0.0)
    if renormalize:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    total = (w * torch.tensor(g)).sum()
    c = None
    if load:
        loss, c = ref.balance_loss(z, ids, score=score, coef=coef)
        q = s / s.sum(1, keepdim=True)
        rows = on.any(1)
        count = torch.bincount(torch.tensor(ids)[on].long(), minlength=E).double()
        lt = coef * E * (count / count.sum() * q[rows].mean(0)).sum()
        np.testing.assert_allclose(loss, lt.item(), rtol=1e-12)
        total = total + 0.7 * lt
    total.backward()
    got, size = ref.select_backward(z, ids, g, score=score, renormalize=renormalize, load=c,
                                    grad_loss=0.7)
    np.testing.assert_allclose(got, zt.grad.numpy(), rtol=1e-9, atol=1e-14)
    assert (np.abs(got) <= size * (1 + 1e-9)).all() and (got[4] == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_by_differences(score):
    z, h = _z(3, 9, 4), 1e-6
    ids, _ = ref.select(z, score=score, topk=3)
    g = np.random.default_rng(5).normal(size=(3, 3))

    def value(z):
        s = np.exp(ref.log_scores(z, score))
        w = np.take_along_axis(s, ids, 1)
        return (g * w / w.sum(1, keepdims=True)).sum()

    got, _ = ref.select_backward(z, ids, g, score=score)
    for t, e in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[t, e] = h
        assert abs((value(z + d) - value(z - d)) / (2 * h) - got[t, e]) < 1e-8


def test_balance_loss_of_an_even_load_is_coef():
    ids = np.arange(16).reshape(8, 2) % 8
    loss, load = ref.balance_loss(np.zeros((8, 8)), ids, coef=0.3)
    np.testing.assert_allclose(loss, 0.3, rtol=1e-14)
    np.testing.assert_allclose(load, 0.3 / 8, rtol=1e-14)
    assert ref.balance_loss(np.zeros((2, 4)), np.full((2, 2), -1))[0] == 0.0


def test_e2m1_values_and_rounding():
    # sign, two exponent bits (bias 1), one mantissa bit
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = m * 0.5 if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
        assert fp4.E2M1[c] == (-v if c & 8 else v)
    w = np.zeros(32)
    w[:12] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.26, 6.9, -0.1]
    codes, scales = fp4.quantize(w)
    assert scales.tolist() == [127]
    assert fp4.dequantize(codes, scales)[:12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4, 0.5, 6, 0]
    # no weight is off by more than half a step of its place
    v = np.random.default_rng(0).normal(size=(50, 64))
    codes, scales = fp4.quantize(v)
    a = np.abs(v) / np.repeat(fp4.scale_value(scales), 32, 1)
    assert a.max() <= 7
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))
    back = np.abs(fp4.dequantize(codes, scales)) / np.repeat(fp4.scale_value(scales), 32, 1)
    assert (np.abs(back - a) <= half + 1e-15).all()


def test_scales_of_extreme_groups():
    w = np.zeros((4, 32))
    w[1, 3] = 2.0 ** -133           # below the least scale's half step
    w[2, 0] = 7.0 * 2.0 ** 10
    w[3, 0] = np.inf
    codes, scales = fp4.quantize(w)
    assert scales[:, 0].tolist() == [1, 1, 137, 255] and not codes[:2].any()
    assert np.isnan(fp4.dequantize(codes, scales)[3]).all()


def test_fragment_order():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, size=(2, 32, 256)).astype(np.uint8)
    scales = rng.integers(0, 256, size=(2, 32, 8)).astype(np.uint8)
    q = fp4.pack_codes(codes).reshape(2, 2, 2, 2, 64, 8)
    s = fp4.pack_scales(scales).reshape(2, 2, 2, 16, 4)
    for _ in range(200):
        e, n, k = rng.integers(2), rng.integers(32), rng.integers(256)
        b, r, t = n // 16, n % 16, k // 128
        step, g, i = k % 128 // 32, k % 32 // 8, k % 8
        byte = q[e, b, t, step // 2, 16 * g + r, 4 * (step % 2) + i // 2]
        assert (byte >> (4 * (i & 1))) & 15 == codes[e, n, k]
        assert s[e, b, t, r, step] == scales[e, n, k // 32]
