"""ctypes binding of the training calls: rows sorted by expert and back with
their gradients, the router's gradient, AdamW, and the router's training loop
made of them.

As in the rest of the binding, every step runs in the library's HIP kernels on
the current stream of the tensors' device; nothing falls back to torch.  Results
have no autograd graph, also where inputs require grad: a call and its gradient
go into the forward and backward of a torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from . import _lib
from ._lib import (DTYPE_BF16, DTYPE_FP32, ENTRY_ROUTE_BACKWARD, LAYOUT_ROW_MAJOR, Fp4Weights,
                   Fp8Weights, MoeAdamw, MoeAdamwTensor, _call, _check, make_config,
                   workspace_bytes)

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}

# A call of these on a small batch takes the GPU less time than the host needs
# for it, so the checks that pass cost as little as they can: one expression
# per tensor, whose failure hands the tensor to _check for the error.


def _at(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape, device):
    """t is a dense tensor of this type and shape on `device`, a HIP device."""
    try:
        good = (t.dtype is dtype and t.shape == shape and t.device == device
                and t.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        _check(t, name, dtype, shape, device)


def _need_rows(t, name, rows=None):
    """(width, type, device) of a dense [rows, H] tensor, bf16 or fp32."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        _check(t, name, t.dtype)
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows):
        want = "T" if rows is None else rows
        raise ValueError(f"{name} must have shape ({want}, H), got {tuple(shape)}")
    return shape[1], t.dtype, t.device


def _launch(name, device, *args):
    """Calls the library on the current stream of the tensors' device,
    whichever device is current."""
    call = getattr(_lib.lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch.cuda.current_device():
        status = call(*args, stream)
    else:
        with torch.cuda.device(device):
            status = call(*args, stream)
    if status:
        _call(name, status)


def _scratch(nbytes, device, workspace):
    """The call's workspace: the caller's, or memory of torch's allocator that
    is given back when the call returns (its next use follows on the stream;
    under capture it is of the graph's own pool)."""
    if workspace is not None:
        return workspace.get(nbytes, device)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _tokens_of(perm_dst, topk):
    """T of perm_dst [T*topk]."""
    if not isinstance(perm_dst, torch.Tensor):
        raise TypeError("perm_dst must be a torch.Tensor")
    if perm_dst.dim() != 1 or topk < 1 or perm_dst.numel() % topk:
        raise ValueError(f"perm_dst must have shape (T * {topk},), got {tuple(perm_dst.shape)}")
    return perm_dst.numel() // topk


# Configurations are values: one object per distinct set of numbers.
@functools.lru_cache(maxsize=256)
def _rows_config(T, H, topk, scale=1.0):
    return ctypes.byref(make_config(T, H, 128, num_groups=1, topk_groups=1, topk=topk,
                                    routed_scaling=scale))


@functools.lru_cache(maxsize=256)
def _route_config(T, H, E, topk, renormalize):
    cfg = make_config(T, H, 128, num_experts=E, num_groups=1, topk_groups=1, topk=topk,
                      renormalize=renormalize)
    return ctypes.byref(cfg), workspace_bytes(cfg, ENTRY_ROUTE_BACKWARD)


def dispatch(x, perm_dst, *, topk=8, topk_w=None, out=None):
    """Tokens sorted by expert: x_perm [T*k, H] with x_perm[perm_dst[t*k + j]] =
    x[t], times topk_w[t, j] (fp32 [T, k]) where that is given.  x is bf16 or
    fp32, of any width.

    Rows that no pair names (as many as perm_dst has entries of -1, the last
    ones of moe_permute's order) are left as ``out`` holds them; without
    ``out`` they are not initialised.  ``out`` overlaps no input."""
    T = _tokens_of(perm_dst, topk)
    H, dt, dev = _need_rows(x, "x", T)
    _need(perm_dst, "perm_dst", torch.int32, (T * topk,), dev)
    if topk_w is not None:
        _need(topk_w, "topk_w", torch.float32, (T, topk), dev)
    if out is None:
        out = torch.empty(T * topk, H, dtype=dt, device=dev)
    else:
        _need(out, "out", dt, (T * topk, H), dev)
    if T:
        _launch("moe_dispatch", dev, _rows_config(T, H, topk), _DTYPES[dt], x.data_ptr(),
                perm_dst.data_ptr(), _at(topk_w), out.data_ptr())
    return out


def dispatch_backward(grad_x_perm, perm_dst, *, topk=8, x=None, topk_w=None):
    """Gradient of dispatch: grad_x [T, H], the (weighted) sum of each token's
    rows of grad_x_perm [T*k, H].  With x and topk_w given, (grad_x,
    grad_topk_w fp32 [T, k]); with topk_w alone, grad_x."""
    T = _tokens_of(perm_dst, topk)
    H, dt, dev = _need_rows(grad_x_perm, "grad_x_perm", T * topk)
    _need(perm_dst, "perm_dst", torch.int32, (T * topk,), dev)
    if topk_w is not None:
        _need(topk_w, "topk_w", torch.float32, (T, topk), dev)
    if x is not None:
        if topk_w is None:
            raise ValueError("x is for the gradient of topk_w: pass topk_w too")
        _need(x, "x", dt, (T, H), dev)
    grad_x = torch.empty(T, H, dtype=dt, device=dev)
    grad_w = None if x is None else torch.empty_like(topk_w)
    if T:
        _launch("moe_dispatch_backward", dev, _rows_config(T, H, topk), _DTYPES[dt],
                grad_x_perm.data_ptr(), perm_dst.data_ptr(), _at(topk_w), _at(x),
                grad_x.data_ptr(), _at(grad_w))
    return grad_x if x is None else (grad_x, grad_w)


def combine_backward(grad_out, y_perm, perm_dst, topk_w, *, routed_scaling=2.5, need_grad_y=True,
                     need_grad_w=True, out=None):
    """Gradient of combine: (grad_y_perm [T*k, H], grad_topk_w fp32 [T, k]);
    None in the place of one that is not needed.  y_perm may be None without
    need_grad_w.  Rows of grad_y_perm that no pair names are left as ``out``
    holds them (without ``out``: not initialised); ``out`` overlaps no input."""
    if not (need_grad_y or need_grad_w):
        raise ValueError("combine_backward: no gradient asked for")
    if not isinstance(topk_w, torch.Tensor) or topk_w.dim() != 2:
        raise TypeError("topk_w must be a torch.Tensor [T, k]")
    T, k = topk_w.shape
    H, dt, dev = _need_rows(grad_out, "grad_out", T)
    _need(perm_dst, "perm_dst", torch.int32, (T * k,), dev)
    _need(topk_w, "topk_w", torch.float32, (T, k), dev)
    if y_perm is not None:
        _need(y_perm, "y_perm", dt, (T * k, H), dev)
    elif need_grad_w:
        raise ValueError("the gradient of topk_w needs y_perm")
    grad_y = grad_w = None
    if need_grad_y:
        if out is None:
            grad_y = torch.empty(T * k, H, dtype=dt, device=dev)
        else:
            _need(out, "out", dt, (T * k, H), dev)
            grad_y = out
    if need_grad_w:
        grad_w = torch.empty_like(topk_w)
    if T:
        _launch("moe_combine_backward", dev, _rows_config(T, H, k, float(routed_scaling)),
                _DTYPES[dt], grad_out.data_ptr(), _at(y_perm), perm_dst.data_ptr(),
                topk_w.data_ptr(), _at(grad_y), _at(grad_w))
    return grad_y, grad_w


def route_backward(x, w_router, topk_ids, topk_logits, grad_topk_w, perm_src, offsets, *,
                   renormalize=True, grad_x_add=None, need_grad_x=True, grad_w_router=None,
                   workspace=None):
    """Gradient of route / route_replay: (grad_w_router fp32 [E, H], grad_x bf16
    [T, H] or None), from the gradient of the combine weights.

    topk_logits is what route(..., return_logits=True) returned; perm_src and
    offsets are permute's for the same ids.  ``grad_x_add`` (bf16 [T, H], the
    hidden state's gradient through the experts) is added into grad_x before
    its one rounding.  A ``grad_w_router`` passed in is added to (gradients of
    several micro-batches) and returned."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a torch.Tensor [T, H]")
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise TypeError("topk_ids must be a torch.Tensor [T, k]")
    if not isinstance(w_router, torch.Tensor) or w_router.dim() != 2:
        raise TypeError("w_router must be a torch.Tensor [E, H]")
    (T, H), k, E, dev = x.shape, topk_ids.shape[1], w_router.shape[0], x.device
    f32, i32, pairs = torch.float32, torch.int32, (T, k)
    if x.dtype is not torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        _check(x, "x", torch.bfloat16)
    _need(w_router, "w_router", f32, (E, H), dev)
    _need(topk_ids, "topk_ids", i32, pairs, dev)
    _need(topk_logits, "topk_logits", f32, pairs, dev)
    _need(grad_topk_w, "grad_topk_w", f32, pairs, dev)
    _need(perm_src, "perm_src", i32, (T * k,), dev)
    _need(offsets, "offsets", i32, (E + 1,), dev)
    if grad_x_add is not None:
        if not need_grad_x:
            raise ValueError("grad_x_add without need_grad_x")
        _need(grad_x_add, "grad_x_add", torch.bfloat16, (T, H), dev)
    accumulate = grad_w_router is not None
    if accumulate:
        _need(grad_w_router, "grad_w_router", f32, (E, H), dev)
    cfg, nb = _route_config(T, H, E, k, bool(renormalize))
    grad_x = torch.empty_like(x) if need_grad_x else None
    if T == 0:
        return (grad_w_router if accumulate else torch.zeros_like(w_router)), grad_x
    if not accumulate:
        grad_w_router = torch.empty_like(w_router)
    ws = _scratch(nb, dev, workspace) if nb else None
    _launch("moe_route_backward", dev, cfg, x.data_ptr(), w_router.data_ptr(),
            topk_ids.data_ptr(), topk_logits.data_ptr(), grad_topk_w.data_ptr(),
            perm_src.data_ptr(), offsets.data_ptr(), _at(grad_x_add), accumulate,
            grad_w_router.data_ptr(), _at(grad_x), _at(ws), nb)
    return grad_w_router, grad_x


# ---------------------------------------------------------------------------
# AdamW
class AdamW:
    """AdamW (decoupled weight decay) over a list of tensors, all updated by one
    call (a launch per 40 tensors).

    params: fp32 tensors, or bf16 ones, which get an fp32 master copy that the
    update works on; contiguous, 16-byte aligned (gradients too), on one device,
    apart in memory, updated in place.  state_bits: 32, or 8 for states in E4M3
    codes with a power-of-two scale per 32 elements (2.06 bytes per element
    instead of 8), rounded stochastically from ``seed``.

    ``state`` is a dict of lists, one entry per parameter: ``exp_avg``,
    ``exp_avg_sq`` (with 8 bits the codes of its square root), with 8 bits
    ``exp_avg_scale`` and ``exp_avg_sq_scale``, and ``master`` (None for fp32
    parameters).  Pass one in, with ``step_count`` (the old one's
    ``step_counts``), to continue from a checkpoint; its tensors are used, not
    copied.

    A parameter without a gradient makes no step, and its bias correction goes
    by the steps that it has made itself.  ``step_counts`` has them, one per
    parameter, and belongs in a checkpoint: ``step_count`` takes such a list,
    or one number for all.

    ``capturable`` keeps the step numbers on the device, so that a captured
    step counts on in each replay."""

    def __init__(self, params, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                 state_bits=32, seed=0, state=None, step_count=0, capturable=False):
        self.params = tuple(params)
        if not self.params:
            raise ValueError("AdamW: no parameters")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        try:
            counts = [operator.index(step_count)] * len(self.params)
        except TypeError:
            counts = [operator.index(c) for c in step_count]
        if len(counts) != len(self.params):
            raise ValueError(f"one step count per parameter ({len(self.params)}) expected, got "
                             f"{len(counts)}")
        if min(counts) < 0:
            raise ValueError("step_count must not be negative")
        first = getattr(self.params[0], "device", None)
        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor) or p.dtype not in _DTYPES:
                raise TypeError(f"params[{i}] must be torch.bfloat16 or torch.float32, got "
                                f"{getattr(p, 'dtype', type(p))}")
            if not (p.is_cuda and p.device == first and p.is_contiguous()):
                _check(p, f"params[{i}]", p.dtype, None, first)
        places = [p.data_ptr() for p in self.params if p.numel()]
        if len(set(places)) < len(places):
            raise ValueError("AdamW: a parameter is listed twice")
        self.device = self.params[0].device
        self.lr, self.state_bits = lr, state_bits
        # steps of the list, and by how many those of a parameter are fewer; on
        # the device the list's number, then every parameter's
        self._steps, self._step_dev = max(counts), None
        self._missed = {i: self._steps - c for i, c in enumerate(counts) if c < self._steps}
        if capturable:
            self._step_dev = torch.tensor([self._steps, *counts], dtype=torch.int64,
                                          device=self.device)
            self._counters = self._step_dev.split(1)
        self.state = self._new_state() if state is None else self._taken(state)
        self._refuse_overlaps()
        self._list = (MoeAdamwTensor * len(self.params))()
        # per parameter: itself, its address, shape, elements, its list entry,
        # the gradient (address, type) that the entry holds, its place
        self._rows = []
        st = self.state
        for i, (p, d) in enumerate(zip(self.params, self._list)):
            d.param, d.master = p.data_ptr(), _at(st["master"][i])
            d.m, d.v = st["exp_avg"][i].data_ptr(), st["exp_avg_sq"][i].data_ptr()
            if state_bits == 8:
                d.m_scale = st["exp_avg_scale"][i].data_ptr()
                d.v_scale = st["exp_avg_sq_scale"][i].data_ptr()
            d.param_dtype, d.state_bits = _DTYPES[p.dtype], state_bits
            if capturable:
                d.step_dev = self._step_dev.data_ptr() + 8 * (i + 1)
            self._rows.append((p, p.data_ptr(), p.shape, p.numel(), d, [None], i))
        # places of the parameters that autograd may have saved for a backward pass
        self._saved = [i for i, p in enumerate(self.params) if p.requires_grad]
        self._opt = MoeAdamw(beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay,
                             seed=seed & 0xFFFFFFFF)
        self._opt_ref = ctypes.byref(self._opt)

    @property
    def step_count(self):
        """Steps made so far (with capturable read from the device)."""
        return self._steps if self._step_dev is None else int(self._step_dev[0])

    @property
    def step_counts(self):
        """The steps that each parameter has made: those with a gradient."""
        if self._step_dev is not None:
            return self._step_dev[1:].tolist()
        return [self._steps - self._missed.get(i, 0) for i in range(len(self.params))]

    def _count(self, absent, by):
        """Adds `by` to the device's step numbers, but for the parameters at the
        places in `absent`."""
        if not absent:
            self._step_dev.add_(by)
        else:
            skip = {i + 1 for i in absent}
            torch._foreach_add_([c for i, c in enumerate(self._counters) if i not in skip], by)

    def _kinds(self):
        """The state's lists and their element types."""
        if self.state_bits == 32:
            return {"exp_avg": torch.float32, "exp_avg_sq": torch.float32}
        return {"exp_avg": torch.float8_e4m3fn, "exp_avg_sq": torch.float8_e4m3fn,
                "exp_avg_scale": torch.float8_e8m0fnu, "exp_avg_sq_scale": torch.float8_e8m0fnu}

    def _new_state(self):
        state = {"master": tuple(p.detach().float() if p.dtype == torch.bfloat16 else None
                                 for p in self.params)}
        for k, dt in self._kinds().items():
            state[k] = tuple(
                torch.zeros((p.numel() + 31) // 32 if k.endswith("scale") else p.shape,
                            dtype=torch.uint8 if dt.itemsize == 1 else dt,
                            device=self.device).view(dt) for p in self.params)
        return state

    def _taken(self, state):
        state = dict(state)
        if "master" not in state and all(p.dtype == torch.float32 for p in self.params):
            state["master"] = [None] * len(self.params)
        kinds = {**self._kinds(), "master": torch.float32}
        if set(state) != set(kinds):
            raise ValueError(f"state must hold {sorted(kinds)}, got {sorted(state)}")
        for k, v in state.items():
            if len(v) != len(self.params):
                raise ValueError(f"state[{k!r}] must have {len(self.params)} entries, got {len(v)}")
            scale = k.endswith("scale")
            for i, (p, t) in enumerate(zip(self.params, v)):
                if k == "master" and p.dtype is torch.float32:
                    if t is not None:
                        raise ValueError(f"state['master'][{i}] must be None: its parameter is "
                                         "fp32")
                    continue
                n = (p.numel() + 31) // 32 if scale else p.numel()
                if (isinstance(t, torch.Tensor) and t.dtype is kinds[k] and t.numel() == n
                        and t.device == self.device and t.is_contiguous()):
                    continue
                _check(t, f"state[{k!r}][{i}]", kinds[k], None, self.device)
                raise ValueError(f"state[{k!r}][{i}] must have {n} elements, got {t.numel()}")
        return {k: tuple(v) for k, v in state.items()}

    def _refuse_overlaps(self):
        """Parameters and states are each written by one workgroup alone: no two
        may share memory."""
        spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name, i)
                 for name, ts in (("params", self.params), *self.state.items())
                 for i, t in enumerate(ts) if t is not None and t.numel()]
        spans.sort()
        for (_, end, name, i), (start, _, other, j) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"AdamW: {name}[{i}] and {other}[{j}] overlap in memory")

    def _pointer(self, t, name):
        """Device address of a one-element fp32 tensor."""
        _check(t, name, torch.float32, None, self.device)
        if t.numel() != 1:
            raise ValueError(f"{name} must have one element, got {t.numel()}")
        return t.data_ptr()

    def _refuse(self, grads):
        """Raises the error of the first gradient or parameter that is wrong."""
        for i, ((p, at, shape, *_), g) in enumerate(zip(self._rows, grads)):
            if g is None:
                continue
            if getattr(g, "dtype", None) not in _DTYPES:
                raise TypeError(f"grads[{i}] must be torch.bfloat16 or torch.float32, got "
                                f"{getattr(g, 'dtype', type(g))}")
            _check(g, f"grads[{i}]", g.dtype, shape, self.device)
            if p.data_ptr() != at:
                raise RuntimeError(f"params[{i}] lies elsewhere than when this AdamW was made: "
                                   "make a new one with its state")

    def step(self, grads, *, lr=None, grad_scale=1.0):
        """One step.  grads: one tensor (bf16 or fp32, the parameter's shape)
        per parameter, or None to leave that parameter, its state and its step
        number alone.
        lr (default: the constructor's) and grad_scale, a factor on every
        gradient, are numbers or one-element fp32 device tensors."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(self.params)} gradients expected, got {len(grads)}")
        dev, opt, index, absent = self.device, self._opt, self.device.index, []
        for (p, at, shape, n, d, held, place), g in zip(self._rows, grads):
            if g is None:
                d.n, held[0] = 0, None
                absent.append(place)
                continue
            try:
                kind = _DTYPES[g.dtype]
                good = (g.shape == shape and g.get_device() == index and g.is_contiguous()
                        and p.data_ptr() == at)
            except (AttributeError, KeyError):
                good = False
            if not good:
                self._refuse(grads)
            entry = (g.data_ptr(), kind)
            if held[0] != entry:
                held[0] = entry
                d.grad, d.grad_dtype, d.n = *entry, n
        if lr is None:
            lr = self.lr
        if isinstance(lr, torch.Tensor):
            opt.lr, opt.lr_dev = 0.0, self._pointer(lr, "lr")
        else:
            opt.lr, opt.lr_dev = float(lr), None
        if isinstance(grad_scale, torch.Tensor):
            opt.grad_scale, opt.grad_scale_dev = 1.0, self._pointer(grad_scale, "grad_scale")
        else:
            opt.grad_scale, opt.grad_scale_dev = float(grad_scale), None
        opt.step = self._steps + 1
        capturing = _lib._capturing(dev)
        if capturing and self._step_dev is None:
            raise RuntimeError("AdamW.step under graph capture needs capturable=True")
        counted = self._step_dev is not None
        if counted:
            self._count(absent, 1)
        else:
            for i, fewer in self._missed.items():
                self._list[i].step = opt.step - fewer
        try:
            _launch("moe_adamw_step", dev, self._opt_ref, self._list, len(self._rows))
        except _lib.MoeError as e:
            if counted:
                self._count(absent, -1)  # refused: no step was made
            for name, ts in (("params", self.params), ("grads", grads)):
                for i, t in enumerate(ts):
                    if t is not None and t.data_ptr() % 16:
                        raise _lib.MoeError(e.code, f"moe_adamw_step: {name}[{i}] is not 16-byte "
                                                    "aligned") from None
            raise
        if not capturing:
            self._steps += 1
            if not counted:
                for i in absent:
                    self._missed[i] = self._missed.get(i, 0) + 1
        if self._saved:  # changed in place: a backward pass that needs the old values fails
            still = set(absent)
            torch.autograd.graph.increment_version(
                [self.params[i] for i in self._saved if i not in still])


# ---------------------------------------------------------------------------
# training the router
class RouterTrainer:
    """Trains a block's router on frozen experts.

    ``forward`` runs the block (route or replay, permute, expert MLPs,
    combine) and keeps what the gradient needs, ``backward`` adds the router's
    gradient of that forward pass to ``grad``, ``step`` is one AdamW step on
    ``w_router`` (fp32 [E, H], in place) and clears ``grad``::

        trainer = RouterTrainer(w_router, w_gate_up, w_down, lr=1e-4)
        for x, target in batches:
            out = trainer.forward(x)
            trainer.backward(loss_gradient(out, target))
            trainer.step()

    Between forward and backward x, w_router and topk_ids stay as they are.  Experts are
    bf16 (w_gate_up, w_down in weight_layout), or Fp8Weights or Fp4Weights in the
    place of w_gate_up with w_down None.  The hidden state's gradient is not computed: it
    would need the experts' own."""

    def __init__(self, w_router, w_gate_up, w_down=None, *, sel_bias=None, num_groups=8,
                 topk_groups=4, topk=8, renormalize=True, routed_scaling=2.5,
                 weight_layout=LAYOUT_ROW_MAJOR, lr=1e-4, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.0, state_bits=32, seed=0):
        self.w_router, self.w_gate_up, self.w_down = w_router, w_gate_up, w_down
        self.sel_bias, self.weight_layout = sel_bias, weight_layout
        self.num_groups, self.topk_groups, self.topk = num_groups, topk_groups, topk
        self.renormalize, self.routed_scaling = renormalize, routed_scaling
        self.optimizer = AdamW([w_router], lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                               state_bits=state_bits, seed=seed)
        self.grad = None
        self._saved = None

    def forward(self, x, topk_ids=None):
        """The block's output bf16 [T, H]; topk_ids replays recorded routing."""
        if topk_ids is None:
            ids, w, z = _lib.route(x, self.w_router, sel_bias=self.sel_bias,
                                   num_groups=self.num_groups, topk_groups=self.topk_groups,
                                   topk=self.topk, renormalize=self.renormalize,
                                   return_logits=True)
        else:
            ids = topk_ids
            w, z = _lib.route_replay(x, self.w_router, ids, renormalize=self.renormalize,
                                     return_logits=True)
        _, offsets, src, dst = _lib.permute(ids, num_experts=self.w_router.shape[0])
        if isinstance(self.w_gate_up, Fp8Weights):
            y = _lib.expert_ffn_fp8(x, src, offsets, self.w_gate_up, topk=ids.shape[1])
        elif isinstance(self.w_gate_up, Fp4Weights):
            y = _lib.expert_ffn_fp4(x, src, offsets, self.w_gate_up, topk=ids.shape[1])
        else:
            y = _lib.expert_ffn(x, src, offsets, self.w_gate_up, self.w_down, topk=ids.shape[1],
                                weight_layout=self.weight_layout)
        self._saved = (x, ids, w, z, offsets, src, dst, y)
        return _lib.combine(y, dst, w, routed_scaling=self.routed_scaling)

    def backward(self, grad_out):
        """Adds the router's gradient for the last forward pass to ``grad``,
        given the gradient of its output (bf16 [T, H])."""
        if self._saved is None:
            raise RuntimeError("RouterTrainer.backward: no forward pass to go back through")
        x, ids, w, z, offsets, src, dst, y = self._saved
        _, grad_w = combine_backward(grad_out, y, dst, w, routed_scaling=self.routed_scaling,
                                     need_grad_y=False)
        self.grad, _ = route_backward(x, self.w_router, ids, z, grad_w, src, offsets,
                                      renormalize=self.renormalize, need_grad_x=False,
                                      grad_w_router=self.grad)
        self._saved = None
        return self.grad

    def step(self, *, lr=None, grad_scale=1.0):
        """One AdamW step on the accumulated gradient, which is then cleared."""
        if self.grad is None:
            raise RuntimeError("RouterTrainer.step: no gradient")
        self.optimizer.step([self.grad], lr=lr, grad_scale=grad_scale)
        self.grad = None
