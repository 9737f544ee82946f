"""Routing from logits and the balance loss on the GPU at their edges: long sums,
and the block's own routing beside them.

U = u(fp32) = 2^-24.  The balance loss's error, counted: a normalised score carries
(28 + 2 D) U of its value, D the spread of its row's logits (as a softmax score of
select does: an exponential, its argument, the sum over the experts, a reciprocal
and a product); a wave's sum of max(16, ceil(T / 128)) / 16 tokens is 64 bits wide
and rounded once (U), 16 of them are added in 32 bits (16 U), the rest is 64 bits and
rounded once (U), as `load` is: (46 + 2 D) U whatever the number of tokens.  coef is
an fp32 argument: where it is no fp32 number (1e-2 is 0.00999999977648258 in fp32,
2.2e-8 = 0.375 U less), both carry U more.
"""
import numpy as np
import pytest
import torch

import grouped_top_routing_amd as gtr
from oracle import scores as ref
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U = 2.0 ** -24


def n64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("T", [2000, 1 << 17, (1 << 23) + 77])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_balance_loss_of_many_like_tokens(T, score):
    """Every token has the same scores, no fractions of a power of two, as a
    collapsed router has: the roundings of a long sum all go one way."""
    say(f"[balance_loss] {T} equal tokens, {score}")
    for gap in (0.4, -1.0, -2.0):
        row = torch.tensor([gap, 0.0])
        z = row.to(DEV).expand(T, 2).contiguous()
        ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
        loss, load = gtr.balance_loss(z, ids, score=score, coef=1.0)
        s = ref.scores(n64(row)[None], score)[0]
        want = 2 * s[0] / s.sum()  # f = (2, 0)
        assert abs(float(loss) - want) <= (46 + 2 * abs(gap)) * U * want, (gap, float(loss), want)
        assert abs(float(load[0]) - 2 / T) <= U * 2 / T and float(load[1]) == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,E", [(200000, 60), (30000, 700), (9000, 8)])
def test_balance_loss_of_many_live_tokens(T, E, score, dt):
    say(f"[balance_loss] {T} tokens of {E}, {score} {dt}")
    g = torch.Generator().manual_seed(T)
    z = (torch.randn(T, E, generator=g) * 1.5).to(dt).to(DEV)
    ids = torch.randint(0, E, (T, 3), generator=g).to(torch.int32)
    loss, load = gtr.balance_loss(z, ids.to(DEV), score=score)
    want, want_load = ref.balance_loss(n64(z), ids.numpy(), score=score)
    D = float((z.amax(1) - z.amin(1)).max())
    assert abs(float(loss) - want) <= (47 + 2 * D) * U * want
    assert (np.abs(n64(load) - want_load) <= 2 * U * want_load).all()


# ---------------------------------------------------------------------------
RULE = dict(num_groups=8, topk_groups=4, topk=8)


def order_gaps(z, bias):
    """By how much the order that the block's rule makes of scores in 64 bits is the
    nearest one, [T]: the smallest gap between neighbours among the nine best experts
    of the kept groups, and between the last kept group and the first that is not."""
    v = ref.scores(z, "sigmoid") + (0.0 if bias is None else bias)
    groups = np.sort(v.reshape(len(v), 8, 32), 2)[:, :, -2:].sum(2)
    rank = np.argsort(-groups, 1, kind="stable")
    total = np.take_along_axis(groups, rank, 1)
    keep = np.zeros_like(groups, bool)
    np.put_along_axis(keep, rank[:, :4], True, 1)
    best = -np.sort(-np.where(np.repeat(keep, 32, 1), v, -np.inf), 1)[:, :9]
    return np.minimum(-np.diff(best, axis=1).max(1), total[:, 3] - total[:, 4])


@pytest.mark.parametrize("T,H", [(1, 256), (37, 512), (700, 1280)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_select_by_the_blocks_rule(T, H, biased):
    """Sigmoids, groups and a bias behind the router GEMM: the reference's choice
    from the call's own logits; route's too, but where scores are nearer than fp32
    tells apart (a sigmoid within 4 U, with a bias 5 U of the value, twice that for
    a pair and again for a group's sum; values below 4 here: 80 U)."""
    say(f"[route_select] T={T} H={H} bias={biased}")
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    W = (torch.randn(256, H, generator=g) * 0.05).to(DEV)
    bias = (torch.randn(256, generator=g) * 0.2).to(DEV) if biased else None
    for renormalize in (True, False):
        kw = dict(sel_bias=bias, renormalize=renormalize, **RULE)
        ids, w, z = gtr.route_select(x, W, score="sigmoid", group_best=2, return_logits=True, **kw)
        want, want_w = ref.select(n64(z), score="sigmoid", group_best=2,
                                  **{**kw, "sel_bias": None if bias is None else n64(bias)})
        assert np.array_equal(ids.cpu().numpy(), want)
        # logits of the chosen are above -8 here: as a renormalised weight of select,
        # (40 + 8 * 8 + 2 * 8) U
        assert np.abs(ref.log_scores(n64(z), "sigmoid")[np.arange(T)[:, None], want]).max() < 8
        assert (np.abs(n64(w) - want_w) <= 120 * U * want_w).all()
        rid, rw = gtr.route(x, W, **kw)
        sure = order_gaps(n64(z), None if bias is None else n64(bias)) > 80 * U
        assert sure.mean() > 0.9
        assert np.array_equal(rid.cpu().numpy()[sure], want[sure])
        assert (np.abs(n64(rw)[sure] - want_w[sure]) <= 120 * U * want_w[sure]).all()


def test_route_and_route_select_at_scores_of_one():
    """Logits from 30 up: every sigmoid is 1 in fp32, by which route orders experts;
    route_select tells groups apart in 64 bits, and experts by their logits."""
    say("[route_select] saturated scores")
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    W = torch.zeros(256, 256, device=DEV)
    W[:, 0] = 30 + torch.arange(256, device=DEV) / 8
    rid, _ = gtr.route(x, W, **RULE)
    assert (rid.cpu() == torch.arange(8)).all()
    ids, w, z = gtr.route_select(x, W, score="sigmoid", return_logits=True, **RULE)
    want, _ = ref.select(n64(z), score="sigmoid", **RULE)
    assert np.array_equal(ids.cpu().numpy(), want) and want[0].min() > 31
    assert torch.equal(w, torch.full_like(w, 0.125))
