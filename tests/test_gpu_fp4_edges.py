"""4-bit expert weights on the GPU at their edges: every code under every scale,
and the rows of a call beside those of another."""
import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
from oracle import fp4
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U, UB = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16
E = 256


def n64(t):
    return t.detach().cpu().double().numpy()


def bf16(a):
    """Rounded once to bf16 (of fp64 values that fp32 holds, or that round alike)."""
    return torch.from_numpy(np.asarray(a)).float().to(BF).double().numpy()


@pytest.fixture(scope="module")
def all_scales():
    """Down weights of one expert, 4096 rows of 256: row n has the scale n / 16 and
    one code, n % 16, that is not 0.  (packed, its row-major value)"""
    H, I = 4096, 256
    n = np.arange(H)
    codes = np.zeros((H, I), np.uint8)
    codes[n, n * 37 % I] = n % 16
    scales = np.repeat((n // 16).astype(np.uint8)[:, None], I // 32, 1)
    u8 = lambda v, *s: torch.full(s, v, dtype=torch.uint8, device=DEV)
    down, sdown = u8(0, E, H, I // 2), u8(127, E, H, I // 32)
    down[5] = torch.from_numpy(fp4.to_bytes(codes)).to(DEV)
    sdown[5] = torch.from_numpy(scales).to(DEV)
    w = gtr.pack_fp4(u8(0, E, 2 * I, H // 2), u8(127, E, 2 * I, H // 32), down, sdown)
    return w, fp4.E2M1[n % 16] * fp4.scale_value(n // 16)


#: pairs of the call (which choose its tiles: 16 rows in two waves or one, 64, 96,
#: 192) and rows of the expert
@pytest.mark.parametrize("pairs,rows", [(8, 3), (700, 20), (2000, 40), (15400, 90), (25700, 180)])
def test_every_code_under_every_scale(all_scales, pairs, rows):
    """2^(s - 127) times each code, for all s: subnormal below 2^-126 (code 0
    and 1 of s), infinite past the largest bf16, NaN for 255.  The activations are
    powers of two, so that an output is one product, rounded once."""
    say(f"[expert_down_fp4] every scale, {pairs} pairs, {rows} rows")
    w, value = all_scales
    weight = bf16(value)
    fits = np.abs(value) < 2.0 ** 128
    assert np.array_equal(weight[fits], value[fits])  # exact in bf16
    assert np.isinf(weight[~fits & ~np.isnan(value)]).all()
    e = np.array([0, 40, -20, 20])[np.arange(rows) % 4]
    h = torch.zeros(pairs, 256, dtype=BF, device=DEV)
    h[:rows] = torch.from_numpy(2.0 ** e)[:, None].to(BF).to(DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[6:] = rows
    y = n64(gtr.expert_down_fp4(h, off, w, topk=1)[:rows])
    want = bf16(weight[None] * (2.0 ** e)[:, None])
    assert np.array_equal(y, want, equal_nan=True)
    tiny = (np.abs(weight) < 2.0 ** -126) & (weight != 0)
    assert tiny.sum() == 8 and (y[1][tiny] != 0).all()


@pytest.mark.parametrize("pairs,rows", [(8, 3), (700, 20), (2000, 40), (15400, 90), (25700, 180)])
def test_a_nan_scale_under_codes_of_one_sign(pairs, rows):
    """NaN, not the infinity that 2^128 would give."""
    say(f"[expert_down_fp4] NaN scale, {pairs} pairs")
    H, I = 256, 128
    u8 = lambda v, *s: torch.full(s, v, dtype=torch.uint8, device=DEV)
    sdown = u8(127, E, H, I // 32)
    sdown[5, 7, 1] = 255
    w = gtr.pack_fp4(u8(0, E, 2 * I, H // 2), u8(127, E, 2 * I, H // 32), u8(0x22, E, H, I // 2),
                     sdown)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[6:] = rows
    y = n64(gtr.expert_down_fp4(torch.ones(pairs, I, dtype=BF, device=DEV), off, w, topk=1)[:rows])
    assert np.isnan(y[:, 7]).all() and (np.delete(y, 7, 1) == I).all()


def test_the_largest_weights(all_scales):
    """7 * 2^125 rounds to 6 * 2^125; the next bf16 number to 4 * 2^126, infinite."""
    say("[quantize_fp4] the largest weights")
    gu, dn = torch.zeros(E, 256, 256, dtype=BF, device=DEV), torch.zeros(E, 256, 128, dtype=BF, device=DEV)
    dn[5, 0, 3], dn[5, 1, 3], dn[5, 2, 3] = 7 * 2.0 ** 125, 7.03125 * 2.0 ** 125, -3.3895e38
    w = gtr.quantize_fp4(gu, dn)
    h = torch.zeros(8, 128, dtype=BF, device=DEV)
    h[:, 3] = 2.0 ** -100
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[6:] = 2
    y = n64(gtr.expert_down_fp4(h, off, w, topk=1)[:2])
    assert (y[:, 0] == 6 * 2.0 ** 25).all() and (y[:, 1] == np.inf).all()
    assert (y[:, 2] == -np.inf).all() and not y[:, 3:].any()


def silu(g):
    return g / (1 + np.exp(-g))


@pytest.mark.parametrize("H,I", [(1024, 512), (2560, 1280)])
def test_rows_alone_and_among_others(H, I):
    """The pairs of a call choose its tiles, and up to 1024 items of 16 rows two
    waves that take half of k each: a token's outputs may differ in their last bits
    from one call to another.  Each call is within the bound of H, then I, roundings
    (U per addition, in any order) and one of each output to bf16; calls that take
    k in one chain agree bit for bit."""
    say(f"[expert_ffn_fp4] rows alone and among others, H={H} I={I}")
    g = torch.Generator(device=DEV).manual_seed(H)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)
    arrays = (r(0, 256, E, 2 * I, H // 2), r(118, 122, E, 2 * I, H // 32),
              r(0, 256, E, H, I // 2), r(118, 122, E, H, I // 32))
    w = gtr.pack_fp4(*arrays)
    k, T = 4, 4000
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
    gate_up, down = {}, {}
    for n in (1, 3, 40, 300, 2000, T):
        _, off, src, dst = gtr.permute(ids[:n].contiguous())
        h = gtr.expert_gate_up_fp4(x[:n], src, off, w, topk=k)
        y = gtr.expert_down_fp4(h, off, w, topk=k)
        assert torch.equal(y, gtr.expert_ffn_fp4(x[:n], src, off, w, topk=k))
        first = dst[:k].long()  # the rows of token 0
        gate_up[n], down[n] = h[first], y[first]
    items = lambda n: (n * k // 16 + min(n * k, E) + 1)
    split = [n for n in gate_up if items(n) * (I // 32) <= 1024 and n * k <= E // 4]
    chain = [n for n in gate_up if items(n) * (I // 32) > 1024 and items(n) * (H // 64) > 1024]
    assert 1 in split and T in chain and 300 in chain
    for n in chain:
        assert torch.equal(gate_up[n], gate_up[T])
    dense = lambda q, s, e: fp4.dequantize(
        np.stack((q[e].cpu().numpy() & 15, q[e].cpu().numpy() >> 4), -1).reshape(q.shape[1], -1),
        s[e].cpu().numpy())
    X = n64(x[0])
    for j, e in enumerate(ids[0].tolist()):
        W, D = dense(*arrays[:2], e), dense(*arrays[2:], e)
        s, mag = W @ X, np.abs(W) @ np.abs(X) * (H * U)
        a, u, da, du = s[:I], s[I:], mag[:I], mag[I:]
        want = silu(a) * u
        bound = 1.1 * np.abs(u) * da + np.abs(a) * du + 1.1 * da * du + (8 * U + UB) * np.abs(want)
        for n in gate_up:
            h = n64(gate_up[n][j])
            assert (np.abs(h - want) <= bound).all(), (n, j)
            y = D @ h
            assert (np.abs(n64(down[n][j]) - y)
                    <= I * U * (np.abs(D) @ np.abs(h)) + UB * np.abs(y)).all(), (n, j)
