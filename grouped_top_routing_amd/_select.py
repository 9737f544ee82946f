"""ctypes binding of routing from logits: selection with softmax or sigmoid
scores, its gradient, and the loss that balances the experts' load.

Every step runs in the library's HIP kernels on the current stream of the
tensors' device.  Results have no autograd graph: a call and its gradient go
into the forward and backward of a torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import (DTYPE_BF16, DTYPE_FP32, ENTRY_ROUTE, MoeError, MoeSelectConfig, _check, lib,
                   make_config, workspace_bytes)
from ._train import _launch, _need, _scratch

SCORES = {"sigmoid": 0, "softmax": 1}
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}

# torch gives an empty tensor no address.  The library reads and writes nothing of an
# empty batch, but checks its arguments as any other's.
_NOWHERE = 256


def _at(t):
    return None if t is None else t.data_ptr() or _NOWHERE


# Configurations are values: one object per distinct set of numbers.
@functools.lru_cache(maxsize=256)
def _config(T, E, k, score, renormalize, dtype, groups=1, topk_groups=1, group_best=2):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return MoeSelectConfig(T, E, groups, topk_groups, group_best, k, SCORES[score],
                           int(bool(renormalize)), _DTYPES[dtype])


@functools.lru_cache(maxsize=256)
def _balance_bytes(T, E, k, score, dtype):
    n = ctypes.c_size_t(0)
    st = lib().moe_balance_workspace_bytes(
        ctypes.byref(_config(T, E, k, score, True, dtype)), ctypes.byref(n))
    if st:
        raise MoeError(st, "moe_balance_workspace_bytes")
    return int(n.value)


def _need_logits(logits):
    """(T, E, type, device) of dense logits [T, E], bf16 or fp32."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in _DTYPES:
        raise TypeError(f"logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must have shape (T, E), got {tuple(logits.shape)}")
    if not logits.is_cuda or not logits.is_contiguous():
        _check(logits, "logits", logits.dtype)
    return (*logits.shape, logits.dtype, logits.device)


def _need_ids(topk_ids, T, device):
    """k of topk_ids [T, k]."""
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise TypeError("topk_ids must be a torch.Tensor [T, k]")
    k = topk_ids.shape[1]
    _need(topk_ids, "topk_ids", torch.int32, (T, k), device)
    return k


def select(logits, *, score="softmax", sel_bias=None, num_groups=1, topk_groups=1, group_best=2,
           topk=8, renormalize=True):
    """Routing from logits [T, E] (bf16 or fp32, up to 1024 experts): (topk_ids
    int32 [T, k], topk_w fp32 [T, k]).

    score: "softmax" over the experts, or "sigmoid".  sel_bias (fp32 [E]) is
    added to the scores for choosing only.  num_groups contiguous groups of
    experts are ranked by the sum of their group_best (1 or 2) largest values
    and the topk_groups best kept.  renormalize: weights over the sum of the
    chosen scores.  Ties go to the lower index.  A logit of -inf (or a bias of
    -inf) masks its expert; slots left without one hold id -1 and weight 0."""
    T, E, dt, dev = _need_logits(logits)
    if sel_bias is not None:
        _need(sel_bias, "sel_bias", torch.float32, (E,), dev)
    cfg = _config(T, E, topk, score, renormalize, dt, num_groups, topk_groups, group_best)
    ids = torch.empty(T, topk, dtype=torch.int32, device=dev)
    w = torch.empty(T, topk, dtype=torch.float32, device=dev)
    _launch("moe_select", dev, ctypes.byref(cfg), _at(logits), _at(sel_bias), _at(ids), _at(w))
    return ids, w


def route_select(x, w_router, *, score="softmax", sel_bias=None, num_groups=1, topk_groups=1,
                 group_best=2, topk=8, renormalize=True, return_logits=False, workspace=None):
    """select on the logits of the block's router (as route computes them in
    FP32 from x bf16 [T, H] and w_router fp32 [256, H]): (topk_ids, topk_w), and
    with return_logits all logits too (fp32 [T, E], for select_backward and
    balance_loss).

    route and layer_forward compare scores in fp32: with sigmoids and groups the
    choice is theirs but where values are nearer than that (scores of 1, say), so
    a router that they are to serve is trained on the ids of route."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a torch.Tensor [T, H]")
    if not isinstance(w_router, torch.Tensor) or w_router.dim() != 2:
        raise TypeError("w_router must be a torch.Tensor [E, H]")
    (T, H), E, dev = x.shape, w_router.shape[0], x.device
    _check(x, "x", torch.bfloat16)
    _need(w_router, "w_router", torch.float32, (E, H), dev)
    if sel_bias is not None:
        _need(sel_bias, "sel_bias", torch.float32, (E,), dev)
    cfg = make_config(T, H, 128, num_experts=E, num_groups=1, topk_groups=1, topk=1)
    sel = _config(T, E, topk, score, renormalize, torch.float32, num_groups, topk_groups,
                  group_best)
    nb = workspace_bytes(cfg, ENTRY_ROUTE)
    ids = torch.empty(T, topk, dtype=torch.int32, device=dev)
    w = torch.empty(T, topk, dtype=torch.float32, device=dev)
    z = torch.empty(T, E, dtype=torch.float32, device=dev) if return_logits else None
    ws = _scratch(nb, dev, workspace)
    _launch("moe_route_select", dev, ctypes.byref(cfg), ctypes.byref(sel), _at(x), _at(w_router),
            _at(sel_bias), _at(ids), _at(w), _at(z), _at(ws), nb)
    return (ids, w, z) if return_logits else (ids, w)


def balance_loss(logits, topk_ids, *, score="softmax", coef=1e-2, workspace=None):
    """The loss coef * sum_e f_e P_e that evens out the experts' load: f_e is
    expert e's share of the pairs times E, P_e its mean score (of the scores
    over their sum) over the rows of logits [T, E] that have an id in [0, E) in
    topk_ids [T, k].

    Returns (loss fp32, load fp32 [E]); load is the loss's derivative by each
    row's scores, which select_backward takes."""
    T, E, dt, dev = _need_logits(logits)
    k = _need_ids(topk_ids, T, dev)
    cfg = _config(T, E, k, score, True, dt)
    nb = _balance_bytes(T, E, k, score, dt)
    new = torch.empty if T else torch.zeros  # the call writes nothing of no tokens
    loss = new((), dtype=torch.float32, device=dev)
    load = new(E, dtype=torch.float32, device=dev)
    ws = _scratch(nb, dev, workspace)
    _launch("moe_balance_loss", dev, ctypes.byref(cfg), _at(logits), _at(topk_ids), float(coef),
            loss.data_ptr(), load.data_ptr(), _at(ws), nb)
    return loss, load


def select_backward(logits, topk_ids, grad_topk_w, *, score="softmax", renormalize=True, load=None,
                    grad_loss=None):
    """Gradient of select's weights with respect to logits: [T, E], of their
    type, dense.  grad_topk_w is fp32 [T, k].

    load (from balance_loss) adds that loss's gradient, times grad_loss (a
    one-element fp32 device tensor; None: 1); grad_topk_w may then be None."""
    T, E, dt, dev = _need_logits(logits)
    k = _need_ids(topk_ids, T, dev)
    if grad_topk_w is not None:
        _need(grad_topk_w, "grad_topk_w", torch.float32, (T, k), dev)
    elif load is None:
        raise ValueError("select_backward: neither grad_topk_w nor load given")
    if load is not None:
        _need(load, "load", torch.float32, (E,), dev)
    if grad_loss is not None:
        if load is None:
            raise ValueError("grad_loss without load")
        _check(grad_loss, "grad_loss", torch.float32, None, dev)
        if grad_loss.numel() != 1:
            raise ValueError(f"grad_loss must have one element, got {grad_loss.numel()}")
    cfg = _config(T, E, k, score, renormalize, dt)
    grad = torch.empty_like(logits)
    _launch("moe_select_backward", dev, ctypes.byref(cfg), _at(logits), _at(topk_ids),
            _at(grad_topk_w), _at(load), _at(grad_loss), _at(grad))
    return grad
