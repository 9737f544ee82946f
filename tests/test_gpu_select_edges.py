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
