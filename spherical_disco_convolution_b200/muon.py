"""The Muon update of the layers' weights, on the libdisco C ABI.

A weight of a DISCO layer is (C_out, C_in / groups, K); the rows of one group are one matrix of
C_out / groups rows and C_in / groups * K columns, and the update of each matrix is made nearly
orthogonal by Newton-Schulz products before it is applied (K. Jordan et al., "Muon: an optimizer
for hidden layers in neural networks", 2024).  Any tensor of two or more axes works the same way,
its first axis the rows.  Everything runs in libdisco's CUDA kernels (there is no CPU path), for
all tensors of one shape together.  fp32 or bf16; momentum is always fp32.
"""

from __future__ import annotations

import functools
import operator

import torch

from . import disco as D
from ._launch import DTYPES, dense, launch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrix(t, groups):
    if t.dim() < 2 or t.numel() == 0:
        raise ValueError(f"a tensor of shape {tuple(t.shape)} is no matrix: two axes or more, none empty")
    if groups <= 0 or t.shape[0] % groups:
        raise ValueError(f"groups={groups} must divide the first axis, {t.shape[0]}")
    return t.shape[0] // groups, t.numel() // t.shape[0]


def _as_list(ts, what):
    if isinstance(ts, torch.Tensor):
        return [ts], True
    ts = list(ts)
    if not ts:
        raise ValueError(f"{what} is an empty list")
    return ts, False


def _buckets(ts):
    """Indices of the tensors that one call can take together."""
    x = ts[0]
    shape, dtype, device = x.shape, x.dtype, x.device
    if all(t.shape == shape and t.dtype == dtype and t.device == device for t in ts):
        return [range(len(ts))]
    by = {}
    for i, t in enumerate(ts):
        by.setdefault((t.shape, t.dtype, t.device), []).append(i)
    return by.values()


_workspace_size = functools.lru_cache(maxsize=1024)(D.disco_orthogonalize_workspace_size)


_cached_rule = functools.lru_cache(maxsize=64)(D.newton_schulz)


def _rule(steps, coefficients, eps):
    a, b, c = coefficients
    return _cached_rule(operator.index(steps), (float(a), float(b), float(c)), float(eps))


def _workspace(x, n, groups, rows, cols):
    """(tensor that holds it, pointer, bytes); small matrices need none."""
    nb = _workspace_size(n, groups, rows, cols)
    if nb == 0:
        return None, None, 0
    ws = x.new_empty(nb, dtype=torch.uint8)
    return ws, ws.data_ptr(), nb


def _outputs(x, n, dtype=None):
    """n tensors like x, each with memory of its own: views of one allocation would share a version
    counter, and an in-place change of one would spoil what autograd saved of the others."""
    return [torch.empty_like(x, dtype=dtype) for _ in range(n)]


def _pointers(ts, what):
    """Pointers of tensors of one bucket, which are dense."""
    if not all([t.is_contiguous() for t in ts]):
        raise ValueError(f"{what} is contiguous")
    return [t.data_ptr() for t in ts]


def _pointers_like(ts, x, what, dtype=None):
    """Pointers of dense tensors of x's shape and device, and of its type or the one given."""
    shape, device, dtype = x.shape, x.device, dtype or x.dtype
    for t in ts:
        if t.dtype != dtype:
            raise TypeError(f"{what} is {dtype} here, not {t.dtype}")
        if t.shape != shape or t.device != device:
            raise ValueError(f"{what} is of shape {tuple(shape)}, on {device}")
    return _pointers(ts, what)


def orthogonalize(update, groups: int = 1, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7):
    """The nearly orthogonal factor of each group's matrix of `update` (one tensor, or a list):
    X = U / (|U| + eps), then `steps` times X <- a X + b (X X^T) X + c (X X^T)^2 X.  It has no gradient."""
    ts, single = _as_list(update, "update")
    ns = _rule(steps, coefficients, eps)
    outs = [None] * len(ts)
    for at in _buckets(ts):
        x = ts[at[0]]
        code = dense(x, "update")
        rows, cols = _matrix(x, groups)
        u = _pointers([ts[i] for i in at], "update")
        out = _outputs(x, len(at))
        ws, p, nb = _workspace(x, len(at), groups, rows, cols)
        launch(x, D.disco_orthogonalize, groups, rows, cols, code, ns, u, [o.data_ptr() for o in out], p, nb)
        for i, o in zip(at, out):
            outs[i] = o
    return outs[0] if single else outs


def _checked(ws, gs, ms, groups):
    """The calls that one step takes, a bucket each: everything but the scalars is checked here,
    before anything is written."""
    calls = []
    for at in _buckets(ws):
        x = ws[at[0]]
        code = dense(x, "weight")
        rows, cols = _matrix(x, groups)
        w = _pointers([ws[i] for i in at], "weight")
        g = _pointers_like([gs[i] for i in at], x, "grad")
        m = _pointers_like([ms[i] for i in at], x, "momentum_buffer", torch.float32)
        _workspace_size(len(at), groups, rows, cols)  # refuses the sizes that the library does not take
        calls.append((at, x, code, rows, cols, w, g, m))
    return calls


def muon_update(weight, grad, momentum_buffer, lr: float, momentum: float = 0.95, nesterov: bool = True,
                weight_decay: float = 0.0, groups: int = 1, steps: int = 5, coefficients=COEFFICIENTS,
                eps: float = 1e-7, inplace: bool = False):
    """(weight', momentum_buffer') of one step (one tensor each, or lists of equal length):
    m' = momentum * m + grad, U = grad + momentum * m' (nesterov) or m', and
    w' = (1 - lr * weight_decay) * w - lr * sqrt(max(1, rows / cols)) * orthogonalize(U).
    momentum_buffer is fp32.  inplace writes both results into the tensors given."""
    ws, single = _as_list(weight, "weight")
    gs, _ = _as_list(grad, "grad")
    ms, _ = _as_list(momentum_buffer, "momentum_buffer")
    if not len(ws) == len(gs) == len(ms):
        raise ValueError(f"{len(ws)} weights, {len(gs)} gradients and {len(ms)} momentum buffers")
    ns = _rule(steps, coefficients, eps)
    calls = _checked(ws, gs, ms, groups)
    if inplace and len({p for c in calls for p in c[5] + c[7]}) < 2 * len(ws):
        raise ValueError("a tensor is given twice: each is updated once")
    w_out, m_out = (ws, ms) if inplace else ([None] * len(ws), [None] * len(ws))
    for at, x, code, rows, cols, w, g, m in calls:
        wp, mp = w, m
        if not inplace:
            wo, mo = _outputs(x, len(at)), _outputs(x, len(at), torch.float32)
            wp, mp = [t.data_ptr() for t in wo], [t.data_ptr() for t in mo]
            for i, a, b in zip(at, wo, mo):
                w_out[i], m_out[i] = a, b
        work, p, nb = _workspace(x, len(at), groups, rows, cols)
        launch(x, D.disco_muon, groups, rows, cols, code, ns, lr, momentum, nesterov, weight_decay, w, g, m, wp, mp, p, nb)
        if inplace:  # a backward pass that kept one of them then raises, as after any in-place operation
            torch.autograd.graph.increment_version([t[i] for t in (ws, ms) for i in at])
    return (w_out[0], m_out[0]) if single else (w_out, m_out)


class Muon(torch.optim.Optimizer):
    """Muon for the weights of DISCO layers (and other parameters of two or more axes).

    A parameter group may set `groups` to its layers' group count.  Vectors (biases, norms) belong
    to another optimizer.  The rate and the other scalars are read at every step, and become
    constants of a CUDA graph that captures it; a first step, which makes the momentum, is not captured."""

    def __init__(self, params, lr: float = 0.02, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, groups: int = 1, steps: int = 5, coefficients=COEFFICIENTS,
                 eps: float = 1e-7):
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay,
                                      groups=groups, steps=steps, coefficients=tuple(coefficients), eps=eps))

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group = self.param_groups[-1]
        try:
            for p in group["params"]:
                _matrix(p, group["groups"])
                if p.dtype not in DTYPES:
                    raise TypeError(f"unsupported dtype {p.dtype}; use float32 or bfloat16")
                if not p.is_contiguous():
                    raise ValueError("Muon takes contiguous parameters")
        except (TypeError, ValueError):
            self.param_groups.pop()
            raise

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        steps = []
        for group in self.param_groups:
            ps = [p for p in group["params"] if p.grad is not None]
            if not ps:
                continue
            for p in ps:
                if "momentum_buffer" not in self.state[p]:
                    if torch.cuda.is_current_stream_capturing():  # a replay would start from zeros every time
                        raise RuntimeError("run one step of Muon before a CUDA graph captures it: it makes the momentum")
                    self.state[p]["momentum_buffer"] = torch.zeros_like(p, dtype=torch.float32)
            steps.append((group, ps, [p.grad.contiguous() for p in ps], [self.state[p]["momentum_buffer"] for p in ps]))
        if len(steps) > 1:  # a group that is refused leaves the others' weights as they were, too
            for group, *tensors in steps:
                _checked(*tensors, group["groups"])
        for group, ps, gs, ms in steps:
            muon_update(ps, gs, ms, group["lr"], group["momentum"], group["nesterov"], group["weight_decay"],
                        group["groups"], group["steps"], group["coefficients"], group["eps"], inplace=True)
        return loss

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        # the base class casts state to the parameter's type; momentum stays fp32
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        params = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(ids, params):
            saved = state_dict["state"].get(i, {}).get("momentum_buffer")
            if saved is not None:
                self.state[p]["momentum_buffer"] = saved.detach().to(device=p.device, dtype=torch.float32, copy=True)
