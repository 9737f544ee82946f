"""CPU-side checks of routing from logits and of the 4-bit expert calls at their
edges: empty batches, and the workspaces' bounds."""
import pytest
import torch

import grouped_top_routing_amd as gtr
from grouped_top_routing_amd import _lib as L
from grouped_top_routing_amd import _select as S

F, I32 = torch.float32, torch.int32


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding's routing calls with CPU tensors taken for a device's: an
    empty batch's call reads no memory and needs no device."""
    monkeypatch.setattr(S, "_need", lambda *a: None)
    monkeypatch.setattr(S, "_check", lambda *a: None)
    monkeypatch.setattr(S, "_need_logits", lambda z: (*z.shape, z.dtype, z.device))

    def launch(name, device, *args):
        status = getattr(gtr.lib(), name)(*args, None)
        if status:
            raise gtr.MoeError(status, name)

    monkeypatch.setattr(S, "_launch", launch)


def z(E=64, T=0, dtype=F):
    return torch.zeros(T, E, dtype=dtype)


def test_empty_batches_give_empty_results(on_cpu):
    ids, w = gtr.select(z(), topk=4, num_groups=8, topk_groups=4, sel_bias=torch.zeros(64))
    assert ids.shape == w.shape == (0, 4)
    loss, load = gtr.balance_loss(z(), ids)
    assert loss.shape == () and load.shape == (64,) and not loss.any() and not load.any()
    for kw in (dict(grad_topk_w=w), dict(grad_topk_w=w, load=load),
               dict(grad_topk_w=None, load=load, grad_loss=torch.ones(()))):
        assert gtr.select_backward(z(), ids, **kw).shape == (0, 64)
    ids, w, logits = gtr.route_select(torch.zeros(0, 256, dtype=torch.bfloat16),
                                      torch.zeros(256, 256), return_logits=True)
    assert ids.shape == w.shape == (0, 8) and logits.shape == (0, 256)


@pytest.mark.parametrize("kw", [dict(topk=100), dict(topk=0), dict(topk=9, num_groups=8),
                                dict(num_groups=7), dict(num_groups=4, topk_groups=5),
                                dict(group_best=3), dict(num_groups=0)])
def test_empty_batches_are_refused_what_others_are(on_cpu, kw):
    with pytest.raises(gtr.MoeError):
        gtr.select(z(), **kw)
    with pytest.raises(gtr.MoeError):
        gtr.route_select(torch.zeros(0, 256, dtype=torch.bfloat16), torch.zeros(256, 256),
                         **({**kw, "topk": 33} if kw.get("topk") == 9 else kw))


def test_empty_batches_of_the_gradient_and_the_loss_are_refused_too(on_cpu):
    ids = lambda k: torch.zeros(0, k, dtype=I32)
    for E, k in ((64, 0), (64, 33), (2000, 8)):
        with pytest.raises(gtr.MoeError):
            gtr.select_backward(z(E), ids(k), torch.zeros(0, k))
        with pytest.raises(gtr.MoeError):
            gtr.balance_loss(z(E), ids(k))
    for coef in (float("nan"), float("inf")):
        with pytest.raises(gtr.MoeError):
            gtr.balance_loss(z(), ids(2), coef=coef)


# ---------------------------------------------------------------------------
def fp4_call(name, topk, groups=8, kept=4):
    """`name` of no tokens on 4-bit experts, hidden 256, intermediate 128."""
    E, H, I = 256, 256, 128
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    w = gtr.Fp4Weights(u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 32), u8(E, H, I // 2),
                       u8(E, H, I // 32))
    x, h = torch.zeros(0, H, dtype=torch.bfloat16), torch.zeros(0, I, dtype=torch.bfloat16)
    src, off = torch.zeros(0, dtype=I32), torch.zeros(E + 1, dtype=I32)
    if name == "layer_forward_fp4":
        return gtr.layer_forward_fp4(x, torch.zeros(E, H), w, topk=topk, num_groups=groups,
                                     topk_groups=kept)
    if name == "expert_down_fp4":
        return gtr.expert_down_fp4(h, off, w, topk=topk)
    return getattr(gtr, name)(x, src, off, w, topk=topk)


@pytest.mark.parametrize("name,width", [("expert_ffn_fp4", 256), ("expert_gate_up_fp4", 128),
                                        ("expert_down_fp4", 256), ("layer_forward_fp4", 256)])
def test_empty_batches_of_4_bit_experts(monkeypatch, name, width):
    monkeypatch.setattr(L, "_check", lambda *a: None)
    assert fp4_call(name, 8).shape == (0, width)
    with pytest.raises(gtr.MoeError):
        fp4_call(name, 9)  # at most 8 slots
    with pytest.raises(gtr.MoeError):
        fp4_call(name, 300)
    if name == "layer_forward_fp4":
        for groups, kept in ((7, 4), (8, 9), (0, 0)):
            with pytest.raises(gtr.MoeError):
                fp4_call(name, 8, groups, kept)


def tile_rows(pairs, weights):
    """Rows per tile of a call of this many pairs on experts of hidden *
    intermediate weights."""
    if pairs <= 64 or pairs <= 1024 and min(pairs, 256) * weights <= 1 << 28:
        return 16
    return 64 if pairs // 256 <= 50 else 96 if pairs // 256 <= 80 else 192


@pytest.mark.parametrize("H,I", [(5120, 2560), (256, 128)])
@pytest.mark.parametrize("k", [1, 8])
def test_fp4_plans_hold_the_worst_split_of_the_pairs(H, I, k):
    """The most tiles that T * k pairs make are one ragged tile for each expert in
    use and whole ones of the rest: the plan has a count (and three words beside
    it) and five words per tile."""
    for T in (0, 1, 2, 7, 8, 9, 31, 64, 128, 129, 1000, 1631, 1632, 2592, 4096, 100000, 1 << 24,
              (1 << 28) - 1):
        n = T * k
        rows = tile_rows(n, H * I)
        # 1 pair each to all experts but one, the rest to that one, or a row more
        # than whole tiles to each
        tiles = [n] if n <= 256 else [255 + -(-(n - 255) // rows)]
        if n > 256:
            each = (n // 256 - 1) // rows * rows + 1
            tiles.append(255 * -(-each // rows) + -(-(n - 255 * each) // rows))
        cfg = gtr.make_config(T, H, I, topk=k, num_groups=1, topk_groups=1,
                              weight_layout=gtr.LAYOUT_FP4_PACKED)
        need = 4 * (4 + 5 * max(tiles))
        assert gtr.workspace_bytes(cfg, gtr.ENTRY_EXPERT_STAGE) >= need, (T, k)
        assert gtr.workspace_bytes(cfg, gtr.ENTRY_EXPERT_FFN) >= need + 2 * n * I, (T, k)
