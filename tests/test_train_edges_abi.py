"""CPU-side checks of the training calls' less usual arguments: each is settled
on the host, before anything reaches a GPU."""
import ctypes

import pytest
import torch

import grouped_top_routing_amd as gtr
from grouped_top_routing_amd import _lib as L
from test_train_abi import A, _opt, _step, _tensor


def test_adamw_checks_the_steps_of_its_tensors():
    for n in (0, 100):
        for kw in (dict(step=-1), dict(step=-(1 << 62)), dict(step_dev=0x10004),
                   dict(step_dev=0x10001)):
            assert _step(_opt(), _tensor(n=n, **kw)) == L.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(step=3), dict(step=(1 << 63) - 1), dict(step_dev=0x10008),
               dict(step=5, step_dev=0x10010)):
        assert _step(_opt(), _tensor(n=0, **kw)) == L.MOE_OK, kw
    # the list has a step of its own in any case
    assert _step(_opt(step=0), _tensor(n=0, step=3)) == L.MOE_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
def test_outputs_that_overlap_are_refused():
    """Every output against every input and every other output: one byte of
    either end in common is refused, side by side passes this check (and then
    finds no device here)."""
    T, H, k, far = 64, 512, 4, 1 << 30
    row, pair = {0: 2 * H, 1: 4 * H}, 4 * T * k
    cfg = gtr.make_config(T, H, 128, num_groups=1, topk_groups=1, topk=k)
    lib, c = gtr.lib(), ctypes.byref(cfg)
    for dt in (0, 1):
        tokens, srt = T * row[dt], T * k * row[dt]
        calls = [
            (lambda *a: lib.moe_dispatch(c, dt, *a, None), [tokens, pair, pair, srt], [3]),
            (lambda *a: lib.moe_dispatch_backward(c, dt, *a, None),
             [srt, pair, pair, tokens, tokens, pair], [4, 5]),
            (lambda *a: lib.moe_combine_rows(c, dt, *a, None), [srt, pair, pair, tokens], [3]),
            (lambda *a: lib.moe_combine_backward(c, dt, *a, None),
             [tokens, srt, pair, pair, srt, pair], [4, 5]),
        ]
        for call, sizes, outs in calls:
            _overlaps(call, sizes, outs, far, set())
    ws = gtr.workspace_bytes(gtr.make_config(300, H, 128, num_groups=1, topk_groups=1, topk=k),
                             gtr.ENTRY_ROUTE_BACKWARD)
    T = cfg.num_tokens = 300
    pair = 4 * T * k
    call = lambda x, w, ids, z, g, src, off, add, gw, gx, work: lib.moe_route_backward(
        c, x, w, ids, z, g, src, off, add, 0, gw, gx, work, ws, None)
    sizes = [T * 2 * H, 1024 * H, pair, pair, pair, pair, 257 * 4, T * 2 * H, 1024 * H, T * 2 * H, ws]
    _overlaps(call, sizes, [8, 9, 10], far, {(9, 7)})


def _overlaps(call, sizes, outs, far, same_is_fine):
    at = [far * (i + 1) for i in range(len(sizes))]
    assert call(*at) == L.MOE_ERR_HIP
    for o in outs:
        for i in range(len(sizes)):
            if i == o:
                continue
            moved = list(at)
            # 16 bytes are the least by which aligned tensors can overlap
            for start in (at[i], at[i] + sizes[i] // 16 * 16 - 16, at[i] - (sizes[o] - 16) // 16 * 16):
                moved[o] = start
                want = (L.MOE_ERR_HIP if (o, i) in same_is_fine and start == at[i]
                        else L.MOE_ERR_INVALID_ARG)
                assert call(*moved) == want, (o, i, start - at[i])
            for start in (at[i] + -(-sizes[i] // 16) * 16, at[i] - -(-sizes[o] // 16) * 16):
                moved[o] = start
                assert call(*moved) == L.MOE_ERR_HIP, (o, i, start - at[i])


def test_route_backward_batches_at_the_grids_limit():
    """The largest batches: of (rows of 256 per expert + experts) * columns / 256
    workgroups, and of tokens * columns / 1024 more where those are launched
    (below 4096 tokens, with grad_x), fewer than 2^24 are taken."""
    def status(T, H, k, gx=A):
        cfg = gtr.make_config(T, H, 128, num_groups=1, topk_groups=1, topk=k)
        # taken: the missing workspace is what is left to refuse
        return gtr.lib().moe_route_backward(ctypes.byref(cfg), A, A, A, A, A, A, A, None, 0, A, gx,
                                            None, 0, None)

    def edge(H, k):
        """The most tokens: (256 + T k / 256) H / 256, a multiple of 8, is below 2^24."""
        rows = ((1 << 24) - 8) // (H // 256) - 256
        return ((rows + 1) * 256 - 1) // k

    for H, k in ((5120, 8), (5120, 3), (7168, 1), (512, 8)):
        T = edge(H, k)
        for gx in (A, None):
            assert status(T, H, k, gx) == L.MOE_ERR_WORKSPACE, (H, k)
            assert status(T + 256, H, k, gx) == L.MOE_ERR_UNSUPPORTED, (H, k)
    # 8 threads per token: fewer than 2^29 tokens
    assert status((1 << 29) - 65, 256, 1) == L.MOE_ERR_WORKSPACE
    assert status(1 << 29, 256, 1) == L.MOE_ERR_UNSUPPORTED
    # few tokens of very many columns
    for T, k in ((129, 1), (4095, 1), (4096, 1)):
        assert status(T, 1 << 24, k, None) == L.MOE_ERR_UNSUPPORTED
    wide = 1 << 22
    assert status(4096, wide, 8) == L.MOE_ERR_WORKSPACE
    assert status(4095, wide, 8) == L.MOE_ERR_UNSUPPORTED
    assert status(4095, wide, 8, None) == L.MOE_ERR_WORKSPACE
    assert status(2000, wide, 8) == L.MOE_ERR_WORKSPACE
    # small batches need no workspace: only the refusal is seen here
    assert status(128, 1 << 24, 8) == L.MOE_ERR_UNSUPPORTED
    assert status(128, (1 << 31) - 256, 8) == L.MOE_ERR_UNSUPPORTED
