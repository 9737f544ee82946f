"""CPU-side checks of the training calls' less usual arguments: each is settled
on the host, before anything reaches a GPU."""
from grouped_top_routing_amd import _lib as L
from test_train_abi import _opt, _step, _tensor


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
