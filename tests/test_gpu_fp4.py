"""4-bit expert weights on the GPU against the plain reference in fp64
(oracle/fp4.py).

Codes, scales and their packed order are equal bit for bit.  Products are exact
(a widened weight has 2 mantissa bits, an activation 8), so a GEMM's only
roundings are its fp32 additions and the one of its output:

* inputs that are small whole numbers, with scales of 2^-1 .. 2^1: every partial
  sum is a multiple of 1/4 below 2^24 / 4, so any order of additions is exact and
  the output is the exact sum rounded once to bf16;
* otherwise an output is within K U of the sum of its terms' magnitudes (U =
  2^-24, K additions), then for gate/up |d(silu(g) u)| <= 1.1 |u| dg + |g| du and
  8 U for the sigmoid, its exponential and the products (exp's argument carries
  none), and u(bf16) = 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
import oracle
from oracle import fp4
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U, UB = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16
E = 256


def n64(t):
    return t.detach().cpu().double().numpy()


def dev(a, dt=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a).astype(dt)).to(DEV)


def routing(counts, T, k, seed=0):
    """Pairs of T tokens dealt to experts with these row counts (sum <= T k; the
    rest are dropped): perm_src, offsets, and the token of each row."""
    counts = np.asarray(counts)
    rng = np.random.default_rng(seed)
    pair = rng.permutation(T * k)[:counts.sum()]
    off = np.zeros(E + 1, np.int64)
    off[1:] = np.cumsum(counts)
    src = np.full(T * k, 2 ** 30)  # entries behind the last row name nothing
    for e in range(E):
        src[off[e]:off[e + 1]] = np.sort(pair[off[e]:off[e + 1]])
    return dev(src), dev(off), src[:off[-1]] // k, off


class Experts:
    """Row-major codes and scales of random experts on the device, and packed."""

    def __init__(self, H, I, seed, whole=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)
        lo, hi = (126, 129) if whole else (118, 124)
        self.gu, self.sgu = r(0, 256, E, 2 * I, H // 2), r(lo, hi, E, 2 * I, H // 32)
        self.dn, self.sdn = r(0, 256, E, H, I // 2), r(lo, hi, E, H, I // 32)
        self.H, self.I = H, I
        self.packed = gtr.pack_fp4(self.gu, self.sgu, self.dn, self.sdn)

    def dense(self, e, down=False):
        q, s = (self.dn, self.sdn) if down else (self.gu, self.sgu)
        b = q[e].cpu().numpy()
        codes = np.stack((b & 15, b >> 4), -1).reshape(b.shape[0], -1)
        return fp4.dequantize(codes, s[e].cpu().numpy())


def silu(g):
    return g / (1 + np.exp(-g))


def bf16(a):
    """Rounded once to bf16 (of exact fp64 values with at most 24 + 8 bits)."""
    return torch.from_numpy(np.asarray(a)).float().to(BF).double().numpy()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,I", [(256, 128), (512, 384), (768, 128)])
def test_quantize_and_pack_are_the_references(H, I):
    say(f"[quantize_fp4] H={H} I={I}")
    g = torch.Generator().manual_seed(H)
    gu = torch.randn(E, 2 * I, H, generator=g) * torch.exp2(
        torch.randint(-20, 20, (E, 2 * I, 1), generator=g).float())
    dn = torch.randn(E, H, I, generator=g)
    # a group of zeros, of ties, of tiny and of huge weights, with an infinity and a NaN
    gu[0, 0, :32] = 0
    gu[0, 1, :32] = torch.tensor([7, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 4) * 2.0 ** -9
    gu[0, 2, :32] = -gu[0, 1, :32]
    gu[0, 3, :32] = 2.0 ** -133
    gu[0, 4, 3] = 2.0 ** 126
    gu[0, 5, 0], gu[0, 6, 31] = float("inf"), float("nan")
    gu, dn = gu.to(BF), dn.to(BF)
    w = gtr.quantize_fp4(gu.to(DEV), dn.to(DEV))
    assert w.shape == (E, H, I) and w.nbytes() == 3 * E * H * I * 17 // 32
    for e in (0, 1, 100, 255):
        for src, q, s in ((gu, w.q_gate_up, w.s_gate_up), (dn, w.q_down, w.s_down)):
            codes, scales = fp4.quantize(src[e].double().numpy())
            keep = np.repeat(scales, 32, 1) != 255
            got_s = s[e].cpu().numpy()
            assert np.array_equal(got_s, fp4.pack_scales(scales))
            got_q = q[e].cpu().numpy()
            same = got_q == fp4.pack_codes(codes)
            assert same.all() or not keep.all() and np.array_equal(
                np.where(fp4.pack_codes((keep * 15).astype(np.uint8)) == 255, got_q, 0),
                np.where(fp4.pack_codes((keep * 15).astype(np.uint8)) == 255,
                         fp4.pack_codes(codes), 0))
    # packing a row-major checkpoint
    rng = np.random.default_rng(H)
    codes = rng.integers(0, 16, (E, 2 * I, H)).astype(np.uint8)
    scales = rng.integers(0, 256, (E, 2 * I, H // 32)).astype(np.uint8)
    cd = rng.integers(0, 16, (E, H, I)).astype(np.uint8)
    sd = rng.integers(0, 256, (E, H, I // 32)).astype(np.uint8)
    d8 = lambda a: dev(a, np.uint8)
    p = gtr.pack_fp4(d8(fp4.to_bytes(codes)), d8(scales), d8(fp4.to_bytes(cd)), d8(sd))
    assert np.array_equal(p.q_gate_up.cpu().numpy(), fp4.pack_codes(codes))
    assert np.array_equal(p.s_gate_up.cpu().numpy(), fp4.pack_scales(scales))
    assert np.array_equal(p.q_down.cpu().numpy(), fp4.pack_codes(cd))
    assert np.array_equal(p.s_down.cpu().numpy(), fp4.pack_scales(sd))


@pytest.fixture(scope="module")
def whole():
    return {}


def whole_experts(cache, H, I):
    if (H, I) not in cache:
        cache.clear()
        cache[H, I] = Experts(H, I, H + I, whole=True)
    return cache[H, I]


#: row counts by expert: none, one, and every count around the row blocks (16)
#: and tiles (32 .. 256) of the kernels
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 159,
         160, 161, 191, 192, 193, 223, 240, 241, 255, 256, 257, 300, 383, 385, 511, 513]


def edge_counts(mean):
    """Row counts of 256 experts: the edges, and a filler that sets the mean (by
    which the calls choose their tiles)."""
    c = np.zeros(E, np.int64)
    c[3:3 + 2 * len(EDGES):2] = EDGES
    left = mean * E - c.sum()
    c[200:] += max(0, left) // 56
    return c


LOADS = {"one": [1] + [0] * 255, "last": [0] * 255 + [7], "few": [2, 0, 1] * 85 + [3],
         "edges": edge_counts(0), "edges, mean 60": edge_counts(60),
         "edges, mean 100": edge_counts(100), "edges, mean 200": edge_counts(200),
         "all to one": [0] * 17 + [1500] + [0] * 238,
         "most to one": [1, 0] * 20 + [800, 17, 0, 33, 64] + [0] * 211, "sixteens": [16] * 256,
         "33 each": [33] * 256}


@pytest.mark.parametrize("load", LOADS)
@pytest.mark.parametrize("H,I", [(256, 128), (512, 384), (1280, 640)])
def test_down_is_the_exact_sum_rounded_once(whole, load, H, I):
    say(f"[expert_down_fp4] {load} H={H} I={I}")
    w = whole_experts(whole, H, I)
    counts = np.asarray(LOADS[load])
    k = 5
    T = -(-counts.sum() // k) + 2  # a few dropped pairs
    _, off_d, _, off = routing(counts, T, k)
    h = torch.randint(-8, 9, (T * k, I), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    h[off[-1]:] = float("nan")  # rows behind the last are not read
    y = gtr.expert_down_fp4(h, off_d, w.packed, topk=k)
    for e in np.nonzero(counts)[0]:
        a, b = off[e], off[e + 1]
        assert np.array_equal(n64(y[a:b]), bf16(n64(h[a:b]) @ w.dense(e, True).T)), e


@pytest.mark.parametrize("load", LOADS)
@pytest.mark.parametrize("H,I", [(256, 128), (768, 256)])
def test_gate_up(load, H, I):
    say(f"[expert_gate_up_fp4] {load} H={H} I={I}")
    w = Experts(H, I, 3)
    counts = np.asarray(LOADS[load])
    k = 4
    T = -(-counts.sum() // k) + 1
    src, off_d, tokens, off = routing(counts, T, k)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    h = gtr.expert_gate_up_fp4(x, src, off_d, w.packed, topk=k)
    worst = 0.0
    for e in np.nonzero(counts)[0]:
        a, b = off[e], off[e + 1]
        X, W = n64(x[torch.from_numpy(tokens[a:b]).to(DEV)]), w.dense(e)
        s, mag = X @ W.T, np.abs(X) @ np.abs(W).T * (H * U)
        g, u, dg, du = s[:, :I], s[:, I:], mag[:, :I], mag[:, I:]
        want = silu(g) * u
        bound = 1.1 * np.abs(u) * dg + np.abs(g) * du + 1.1 * dg * du + (8 * U + UB) * np.abs(want)
        err = np.abs(n64(h[a:b]) - want)
        worst = max(worst, float((err / np.maximum(bound, 1e-300)).max()))
        assert (err <= bound).all(), (e, worst)
    say(f"  largest error {worst:.3f} of its bound")


@pytest.mark.parametrize("T,k", [(1, 8), (1, 1), (2, 8), (32, 8), (100, 3), (700, 8), (3000, 8),
                                 (8000, 8)])
def test_ffn_is_its_halves_and_the_layer_its_steps(T, k):
    say(f"[expert_ffn_fp4] T={T} k={k}")
    H, I = 512, 256
    w = Experts(H, I, 9).packed
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    wr = (torch.randn(E, H, generator=g) * 0.05).to(DEV)
    ids, tw = gtr.route(x, wr, topk=k)
    _, off, src, dst = gtr.permute(ids)
    y = gtr.expert_ffn_fp4(x, src, off, w, topk=k)
    h = gtr.expert_gate_up_fp4(x, src, off, w, topk=k)
    assert torch.equal(y, gtr.expert_down_fp4(h, off, w, topk=k))
    out, li, lw = gtr.layer_forward_fp4(x, wr, w, topk=k, return_routing=True)
    assert torch.equal(li, ids) and torch.equal(lw, tw)
    assert torch.equal(out, gtr.combine(y, dst, tw))
    # any grid, any number of calls: the same bits
    assert torch.equal(y, gtr.expert_ffn_fp4(x, src, off, w, topk=k))


def test_results_do_not_depend_on_the_grid(monkeypatch):
    say("[expert_ffn_fp4] grids")
    for T in (3, 300, 4000):
        w = Experts(256, 128, 2).packed
        x = torch.randn(T, 256, generator=torch.Generator().manual_seed(T)).to(BF).to(DEV)
        ids = dev(np.argsort(np.random.default_rng(T).random((T, E)), 1)[:, :8])
        _, off, src, _ = gtr.permute(ids)
        want = gtr.expert_ffn_fp4(x, src, off, w)
        for n in ("1", "16", "40"):
            monkeypatch.setenv("BEAM_MOE_MAX_GRID", n)
            assert torch.equal(gtr.expert_ffn_fp4(x, src, off, w), want)
        monkeypatch.delenv("BEAM_MOE_MAX_GRID")


def test_rows_behind_the_last_stay(whole):
    say("[expert_ffn_fp4] dropped pairs")
    w = Experts(256, 128, 4).packed
    for T in (5, 900):
        x = torch.randn(T, 256, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
        ids = np.argsort(np.random.default_rng(0).random((T, E)), 1)[:, :8].astype(np.int32)
        ids[np.random.default_rng(1).random((T, 8)) < 0.4] = -1
        _, off, src, dst = gtr.permute(dev(ids))
        n = int(off[-1])
        start = torch.randn(T * 8, 256, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
        y = gtr.expert_ffn_fp4(x, src, off, w, out=start.clone())
        assert torch.equal(y[n:], start[n:]) and not torch.equal(y[:n], start[:n])
        none = torch.full((T, 8), -1, dtype=torch.int32, device=DEV)
        _, off, src, dst = gtr.permute(none)
        assert torch.equal(gtr.expert_ffn_fp4(x, src, off, w, out=start.clone()), start)


def test_extreme_scales_and_infinite_inputs():
    """A NaN scale reaches its own output columns alone; scales at both ends."""
    say("[expert_down_fp4] extreme scales")
    H, I = 256, 128
    w = Experts(H, I, 5, whole=True)
    w.sdn[7, 17, 2], w.sdn[7, 18] = 255, 0
    w.sdn[7, 19], w.sdn[7, 20] = 1, 240
    w.dn[7, 20] = 0x22  # ones
    p = gtr.pack_fp4(w.gu, w.sgu, w.dn, w.sdn)
    for rows in (3, 40, 700):
        counts = np.zeros(E, np.int64)
        counts[7] = rows
        _, off_d, _, off = routing(counts, rows, 1)
        h = torch.ones(rows, I, dtype=BF, device=DEV)
        y = n64(gtr.expert_down_fp4(h, off_d, p, topk=1))
        D = w.dense(7, True)
        assert np.isnan(y[:, 17]).all() and np.isfinite(np.delete(y, 17, 1)).all()
        assert (y[:, 20] == I * 2.0 ** 113).all()
        # scales of 2^-127 and 2^-126: sums below 2^-114, as they are or flushed
        assert (np.abs(y[:, 18:20]) <= 2.0 ** -114).all()
        rest = [c for c in range(H) if c not in (17, 18, 19, 20)]
        assert np.array_equal(y[:, rest], bf16(np.ones((rows, I)) @ D[rest].T))
        h[1, 5] = float("inf")
        y2 = n64(gtr.expert_down_fp4(h, off_d, p, topk=1))
        assert np.array_equal(np.delete(y2, 1, 0), np.delete(y, 1, 0), equal_nan=True)


def test_weights_past_four_gibibytes():
    """The last experts' fragments lie past 2^32 bytes of codes."""
    say("[expert_down_fp4] past 4 GiB")
    H, I = 256 * 40, 128 * 56
    codes = torch.randint(0, 256, (E, H, I // 2), device=DEV, dtype=torch.uint8)
    scales = torch.randint(126, 129, (E, H, I // 32), device=DEV, dtype=torch.uint8)
    assert codes.numel() > 1 << 33
    lib, cfg = gtr.lib(), gtr.make_config(0, H, I, num_groups=1, topk_groups=1, topk=1)
    import ctypes
    q, s = torch.empty_like(codes), torch.empty_like(scales)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    st = torch.cuda.current_stream().cuda_stream
    assert lib.moe_pack_fp4(ctypes.byref(cfg), None, None, ptr(codes), ptr(scales), None, None,
                            ptr(q), ptr(s), ctypes.c_void_p(st)) == 0
    for rows in (2, 70):
        counts = np.zeros(E, np.int64)
        counts[[0, 130, 255]] = rows
        _, off_d, _, off = routing(counts, 3 * rows, 1)
        h = torch.randint(-2, 3, (3 * rows, I), device=DEV).to(BF)
        y = torch.zeros(3 * rows, H, dtype=BF, device=DEV)
        cfg = gtr.make_config(3 * rows, H, I, num_groups=1, topk_groups=1, topk=1,
                              weight_layout=gtr.LAYOUT_FP4_PACKED)
        nb = gtr.workspace_bytes(cfg, gtr.ENTRY_EXPERT_STAGE)
        ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
        assert lib.moe_expert_down_fp4(ctypes.byref(cfg), ptr(h), ptr(off_d), ptr(q), ptr(s),
                                       ptr(y), ptr(ws), nb, ctypes.c_void_p(st)) == 0
        for e in (0, 130, 255):
            b = codes[e].cpu().numpy()
            D = fp4.dequantize(np.stack((b & 15, b >> 4), -1).reshape(H, I),
                               scales[e].cpu().numpy())
            a, z = off[e], off[e + 1]
            assert np.array_equal(n64(y[a:z]), bf16(n64(h[a:z]) @ D.T)), (rows, e)


def test_captured_calls_replay():
    say("[graph] two graphs of the layer on two streams, replayed")
    H, I = 512, 256
    w = Experts(H, I, 6).packed
    g = torch.Generator().manual_seed(0)
    wr = (torch.randn(E, H, generator=g) * 0.05).to(DEV)
    xs = [torch.randn(T, H, generator=g).to(BF).to(DEV) for T in (1, 300)]
    graphs, outs = [], []
    for x in xs:
        gtr.layer_forward_fp4(x, wr, w)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(gtr.layer_forward_fp4(x, wr, w))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for x in xs:
            x.copy_(torch.randn(*x.shape, generator=g).to(BF))
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for x, out in zip(xs, outs):
            assert torch.equal(out, gtr.layer_forward_fp4(x, wr, w)), i
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 37, 128, 700, 3000, 9000])
def test_checked_build_is_silent_and_bitwise_equal(T):
    say(f"[checked] layer_forward_fp4 T={T}")
    H, I = 256, 128
    w = Experts(H, I, 8).packed
    g = torch.Generator().manual_seed(T)
    x, wr = torch.randn(T, H, generator=g).to(BF).to(DEV), torch.randn(E, H, generator=g).to(DEV)
    want = gtr.layer_forward_fp4(x, wr, w)
    torch.cuda.synchronize()
    with gtr.use_library(gtr.LIB_CHECKED_PATH):
        gtr.check_flags()
        got = gtr.layer_forward_fp4(x, wr, w)
        flags = gtr.check_flags()
    assert not any(flags.values()), flags
    assert torch.equal(got, want)


def test_router_trainer_on_4_bit_experts():
    say("[trainer] Fp4Weights")
    T, H, I = 90, 256, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    wr = (torch.randn(E, H, generator=g) * 0.05).to(DEV)
    w = Experts(H, I, 1).packed
    trainer = gtr.RouterTrainer(wr.clone(), w, lr=1e-2)
    out = trainer.forward(x)
    assert torch.equal(out, gtr.layer_forward_fp4(x, wr, w))
    ids, _, z = gtr.route(x, wr, return_logits=True)
    _, off, src, dst = gtr.permute(ids)
    y = gtr.expert_ffn_fp4(x, src, off, w)
    go = torch.randn(T, H, generator=g).to(BF).to(DEV)
    _, gw = gtr.combine_backward(go, y, dst, gtr.route(x, wr)[1], need_grad_y=False)
    want, _ = gtr.route_backward(x, wr, ids, z, gw, src, off, need_grad_x=False)
    assert torch.equal(trainer.backward(go), want)
    trainer.step()
    assert not torch.equal(trainer.w_router, wr)


def test_empty_batches():
    say("[empty] no tokens")
    w = Experts(256, 128, 1).packed
    x = torch.zeros(0, 256, dtype=BF, device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    assert gtr.expert_ffn_fp4(x, i, off, w).shape == (0, 256)
    assert gtr.expert_gate_up_fp4(x, i, off, w).shape == (0, 128)
    assert gtr.expert_down_fp4(torch.zeros(0, 128, dtype=BF, device=DEV), off, w).shape == (0, 256)
    out, ids, tw = gtr.layer_forward_fp4(x, torch.zeros(E, 256, device=DEV), w, return_routing=True)
    assert out.shape == (0, 256) and ids.shape == (0, 8)
