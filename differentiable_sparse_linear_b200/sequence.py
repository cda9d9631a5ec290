"""Sequence operators of libsla: the gated linear recurrence and the routing of tokens to experts.

Both are sparse matrices that a sequence model applies to its tokens, with their transposes and
the gradients on their stored entries, as the rest of the package has them for SPD systems:

``recurrence(a, b, h0, seq_off, gate=...)`` is differentiable: h_t = a_t h_{t-1} + w_t b_t over packed
sequences (the solve with a unit lower bidiagonal matrix); ``sla_recur_solve``, ``sla_recur_adjoint``
and ``sla_recur_step`` are the calls under it and the single-token step on a pool of states.

``sla_route_sort`` sorts tokens by expert into a ``Route``; ``route_dispatch`` (R^T x) and
``route_combine`` (R y) are differentiable in the rows and the weights, over ``sla_route_dispatch``,
``sla_route_combine`` and their adjoints.

Rows are [tokens, channels] tensors of float32, float64, bfloat16 or float16 whose channels are
contiguous; rows may be strided, and an input's rows may be one row expanded.  States, weights
and their gradients are float32 (float64 with float64 rows).  The work runs on the current
stream of the tensors' device, or on ``stream``, in whose memory pool outputs and scratch memory
are then allocated.  Outputs must not share memory with inputs or with each other (different columns of
one buffer do not).

Nothing synchronises, and every call can be captured into a CUDA graph; a graph's scratch memory
belongs to its own pool, so graphs may be replayed at the same time.  A captured backward pass must not
share leaves with an eager graph that is still alive: torch's engine would join the eager
stream, and the capture fails with an error.  Drop the eager graph first, or capture over
``detach().requires_grad_()`` of the leaves.
"""
from __future__ import annotations

import importlib.util
import os
from dataclasses import dataclass
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib

__all__ = [
    "GATES", "Route", "recurrence", "sla_recur_solve", "sla_recur_adjoint", "sla_recur_step",
    "sla_route_sort", "sla_route_dispatch", "sla_route_combine", "sla_route_dispatch_adjoint",
    "sla_route_combine_adjoint", "route_dispatch", "route_combine",
]

# what the stored coefficients hold (SLA_GATE_*): the value, its logarithm, or a sigmoid's argument
GATES = {"value": 0, "exp": 1, "sigmoid": 2}

NATIVE_PATH = os.path.join(_lib.PKG, "lib", "_sla_seq.so")
_native = None


def _load():
    """The native side (csrc/seq_binding.cpp): checks, allocation and the library call.  Loaded at first use;
    there is no other path."""
    global _native
    if _native is None:
        _lib.load()
        if not os.path.exists(NATIVE_PATH):
            raise ImportError(f"_sla_seq.so not found at {NATIVE_PATH}: build it with "
                              "`python -m differentiable_sparse_linear_b200.build`")
        spec = importlib.util.spec_from_file_location("_sla_seq", NATIVE_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        from . import SlaError
        module.set_error_types(SlaError, torch.OutOfMemoryError)
        _native = module
    return _native


def _on(stream, tensor: torch.Tensor):
    """`stream` (a torch stream or a handle) as the current stream of the tensor's device."""
    if not isinstance(tensor, torch.Tensor) or not tensor.is_cuda:
        raise ValueError("libsla takes CUDA tensors")
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = (torch.cuda.ExternalStream(handle, device=tensor.device) if handle
                  else torch.cuda.default_stream(tensor.device))
    if stream.device != tensor.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {tensor.device}")
    return torch.cuda.stream(stream)


def _walkable(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t, or a contiguous copy where no single stride walks its rows."""
    return t if t is None or _load().stride_of(t) is not None else t.contiguous()


# ------------------------------------------------------------------------------ recurrence

def sla_recur_solve(a: torch.Tensor, b: torch.Tensor, h0: Optional[torch.Tensor] = None,
                    seq_off: Optional[torch.Tensor] = None, *, gate: str = "value",
                    out: Optional[torch.Tensor] = None, h_last: Optional[torch.Tensor] = None, stream=None):
    """h_t = a_t h_{t-1} + w_t b_t over every sequence; returns (h, last states).

    a, b: [tokens, channels] packed rows, sequence s owning rows seq_off[s] to seq_off[s + 1] (int32,
    on the device; None: one sequence), or [batch, tokens, channels] sequences of one length.
    gate: what a holds ("value": a itself; "exp": its logarithm; "sigmoid": a = sigmoid, and the
    input is weighted by 1 - a).  h0: [sequences, channels] first states (None: zero).  Rows in no
    sequence come back as zeros, or, with `out` given, as they were."""
    if stream is not None:
        with _on(stream, b):
            return _load().recur_solve(a, b, h0, seq_off, gate, out, h_last)
    return (_native or _load()).recur_solve(a, b, h0, seq_off, gate, out, h_last)


def sla_recur_adjoint(a: torch.Tensor, h: torch.Tensor, dh: Optional[torch.Tensor], *,
                      b: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                      seq_off: Optional[torch.Tensor] = None, dh_last: Optional[torch.Tensor] = None,
                      gate: str = "value", want_da: bool = True, want_db: bool = True,
                      da: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None, stream=None):
    """Adjoint of sla_recur_solve: (dL/da, dL/db, dL/dh0) from dh = dL/dh and dh_last = dL/d(last
    states), either of them None for zero.  h: the rows the solve returned; a, h0, seq_off, gate: as
    there; b: its inputs, which the sigmoid gate's dL/da needs.  dL/da is with respect to what a
    holds.  Skipped gradients (want_da, want_db; dL/dh0 without h0) are None; rows in no sequence
    have zero gradients (with `da`, `db` given they stay as they were)."""
    if stream is not None:
        with _on(stream, h):
            return _load().recur_adjoint(a, h, dh, b, h0, seq_off, dh_last, gate, want_da, want_db, da, db)
    return (_native or _load()).recur_adjoint(a, h, dh, b, h0, seq_off, dh_last, gate, want_da, want_db, da, db)


def sla_recur_step(a: torch.Tensor, b: torch.Tensor, state: torch.Tensor, index: Optional[torch.Tensor] = None, *,
                   gate: str = "value", out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token for each row of a serving batch: state[index[r]] = a_r state[index[r]] + w_r b_r in
    place; returns the new states' rows in b's type.  a, b: [rows, channels]; state: [slots,
    channels] float32 (float64); index: int32 [rows], distinct (None: row r has slot r).  Rows whose
    index is outside the pool are padding: no state changes, and they come back as zeros (with
    `out` given, as they were)."""
    if stream is not None:
        with _on(stream, b):
            return _load().recur_step(a, b, state, index, gate, out)
    return (_native or _load()).recur_step(a, b, state, index, gate, out)


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, h0, seq_off, gate):
        a, b = _walkable(a), _walkable(b)
        h0 = None if h0 is None else h0.contiguous()
        h, last = sla_recur_solve(a, b, h0, seq_off, gate=gate)
        ctx.gate = gate
        ctx.set_materialize_grads(False)
        keep_b = gate == "sigmoid" and ctx.needs_input_grad[0]
        ctx.save_for_backward(a, b if keep_b else None, h, h0, seq_off)
        return h, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dlast):
        if dh is None and dlast is None:
            return None, None, None, None, None
        a, b, h, h0, seq_off = ctx.saved_tensors
        need_a, need_b, need_h0 = ctx.needs_input_grad[:3]
        da, db, dh0 = sla_recur_adjoint(a, h, _walkable(dh), b=b, h0=h0, seq_off=seq_off,
                                        dh_last=None if dlast is None else dlast.contiguous(), gate=ctx.gate,
                                        want_da=need_a, want_db=need_b)
        return da, db, (dh0 if need_h0 else None), None, None


def recurrence(a: torch.Tensor, b: torch.Tensor, h0: Optional[torch.Tensor] = None,
               seq_off: Optional[torch.Tensor] = None, *, gate: str = "value"):
    """(h, last states) of sla_recur_solve, differentiable in a, b and h0.

    The backward pass is one sla_recur_adjoint; it reads h as it was returned, in its own type.
    Inputs whose rows no single stride walks are copied first."""
    return _Recurrence.apply(a, b, h0, seq_off, gate)


# ------------------------------------------------------------------------------ routing

@dataclass
class Route:
    """A routing plan (sla_route_sort).  offsets: [experts + 1] first slot of each expert, the last one
    the number of slots in use; counts: [experts] entries of each expert; entry: [slots] token *
    top_k + choice of a slot, -1 in padding; slot: [tokens, top_k] the inverse, -1 where dropped.
    All int32."""
    offsets: torch.Tensor
    counts: torch.Tensor
    entry: torch.Tensor
    slot: torch.Tensor

    @property
    def n_slots(self) -> int:
        return self.entry.shape[0]


def sla_route_sort(expert: torch.Tensor, n_experts: int, *, align: int = 1, n_slots: Optional[int] = None,
                   stream=None) -> Route:
    """The plan that sorts tokens by expert.  expert: [tokens, top_k] (or [tokens]) int32 or int64 ids;
    ids outside [0, n_experts) are dropped.  Within an expert the order is that of the tokens (and
    choices).  Every expert's slots are padded to a multiple of `align` (a product's tile).
    n_slots: slots to provide (default, and least: tokens * top_k + n_experts * (align - 1))."""
    if stream is not None:
        with _on(stream, expert):
            return Route(*_load().route_sort(expert, n_experts, align, n_slots))
    return Route(*(_native or _load()).route_sort(expert, n_experts, align, n_slots))


def _to_slots(x, route, weight, ys, out, stream):
    if stream is not None:
        with _on(stream, x):
            return _to_slots(x, route, weight, ys, out, None)
    return (_native or _load()).route_to_slots(x, route.offsets, route.counts, route.entry, route.slot, weight, ys, out)


def _to_tokens(ys, route, weight, x, out, stream):
    if stream is not None:
        with _on(stream, ys):
            return _to_tokens(ys, route, weight, x, out, None)
    return (_native or _load()).route_to_tokens(ys, route.offsets, route.counts, route.entry, route.slot, weight, x, out)


def sla_route_dispatch(x: torch.Tensor, route: Route, weight: Optional[torch.Tensor] = None, *,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """xs = R^T x: every slot gets its token's row (times its weight), padding slots zeros.  x:
    [tokens, channels]; weight: [tokens, top_k] float32 (float64) or None for 1.  Slots behind the
    last expert's come back as zeros, or, with `out` given, as they were."""
    return _to_slots(x, route, weight, None, out, stream)[0]


def sla_route_combine_adjoint(dy: torch.Tensor, route: Route, ys: Optional[torch.Tensor] = None,
                              weight: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
                              stream=None):
    """Adjoint of sla_route_combine: (dL/dys = R^T dy, dL/dweight = dy . ys on R's pattern); the
    latter with ys given, else None.  Dropped entries have weight gradient 0."""
    return _to_slots(dy, route, weight, ys, out, stream)


def sla_route_combine(ys: torch.Tensor, route: Route, weight: Optional[torch.Tensor] = None, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = R ys: every token's sum over its slots, times their weights ([tokens, top_k] float32 or
    float64; None: 1), in the order of the choices; a token without slots gets zeros.
    ys: [slots, channels]; rows of slots without an entry are not read."""
    return _to_tokens(ys, route, weight, None, out, stream)[0]


def sla_route_dispatch_adjoint(dxs: torch.Tensor, route: Route, x: Optional[torch.Tensor] = None,
                               weight: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
                               stream=None):
    """Adjoint of sla_route_dispatch: (dL/dx = R dxs, dL/dweight = x . dxs on R's pattern); the
    latter with x given, else None.  Dropped entries have weight gradient 0."""
    return _to_tokens(dxs, route, weight, x, out, stream)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, route):
        x = _walkable(x)
        weight = None if weight is None else weight.contiguous()
        ctx.route = route
        keep_x = weight is not None and ctx.needs_input_grad[1]
        ctx.save_for_backward(x if keep_x else None, weight, route.slot)
        return sla_route_dispatch(x, route, weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        x, weight, _ = ctx.saved_tensors
        dx, dw = sla_route_dispatch_adjoint(_walkable(dxs), ctx.route, x, weight)
        return dx, dw, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weight, route):
        ys = _walkable(ys)
        weight = None if weight is None else weight.contiguous()
        ctx.route = route
        keep_ys = weight is not None and ctx.needs_input_grad[1]
        ctx.save_for_backward(ys if keep_ys else None, weight, route.slot)
        return sla_route_combine(ys, route, weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weight, _ = ctx.saved_tensors
        dys, dw = sla_route_combine_adjoint(_walkable(dy), ctx.route, ys, weight)
        return dys, dw, None


def route_dispatch(x: torch.Tensor, route: Route, weight: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sla_route_dispatch, differentiable in x and weight."""
    return _Dispatch.apply(x, weight, route)


def route_combine(ys: torch.Tensor, route: Route, weight: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sla_route_combine, differentiable in ys and weight."""
    return _Combine.apply(ys, weight, route)
