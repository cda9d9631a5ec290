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
are then allocated.  Nothing synchronises; every call can be captured into a CUDA graph, and a
graph's scratch memory belongs to its own pool.  Inside a capture use the sla_* calls or
``torch.autograd.grad`` on tensors made inside it: ``backward()`` onto leaves that an eager
graph still holds makes torch's engine join that graph's stream, which a capture cannot do.
"""
from __future__ import annotations

import functools
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
_ROW_CODES = {torch.float32: _lib.SLA_F32, torch.float64: _lib.SLA_F64, torch.bfloat16: _lib.SLA_BF16,
              torch.float16: _lib.SLA_F16}


def _check(status: int, where: str) -> None:
    if status < 0:
        from . import SlaError
        raise SlaError(status, where)


def _placed(fn):
    """Runs fn with its first tensor's device current, on that device's current stream or on `stream`."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else next(iter(kw.values()), None)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError("libsla takes CUDA tensors")
        device = first.device
        if stream is None and device.index == torch.cuda.current_device():
            return fn(*args, **kw)
        with torch.cuda.device(device):
            if stream is None:
                return fn(*args, **kw)
            if not isinstance(stream, torch.cuda.Stream):
                handle = int(getattr(stream, "cuda_stream", stream))
                stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                          else torch.cuda.default_stream(device))
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
    return call


def _current(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _code(t: torch.Tensor) -> int:
    code = _ROW_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"rows must be float32, float64, bfloat16 or float16, got {t.dtype}")
    return code


def _wide(dtype: torch.dtype) -> torch.dtype:
    return torch.float64 if dtype == torch.float64 else torch.float32


def _gate(gate: str) -> int:
    code = GATES.get(gate)
    if code is None:
        raise ValueError(f"gate must be one of {sorted(GATES)}, got {gate!r}")
    return code


def _stride(t: torch.Tensor) -> Optional[int]:
    """The one stride that walks t's rows ([rows, channels] or [batch, rows, channels]); None if
    there is none."""
    shape, strides = t.shape, t.stride()
    d = shape[-1]
    if d > 1 and strides[-1] != 1:
        return None
    if len(shape) == 3:
        if shape[0] == 1 or shape[1] == 1:
            ld, n = (strides[1], shape[1]) if shape[0] == 1 else (strides[0], shape[0])
        else:
            ld, n = strides[1], 2
            if strides[0] != shape[1] * ld:
                return None
    else:
        ld, n = strides[0], shape[0]
    if n <= 1:
        return d
    return ld if ld >= d or ld == 0 else None


def _rows(t: torch.Tensor, like: torch.Tensor, name: str, out: bool = False) -> int:
    """Checks rows `t` against `like` (shape, type, device); their row stride."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be {tuple(like.shape)} {like.dtype} on {like.device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    ld = _stride(t)
    if ld is None:
        raise ValueError(f"{name}: channels must be contiguous and rows one stride apart")
    if out and ld < t.shape[-1]:
        raise ValueError(f"{name}: an output's rows must not overlap")
    return ld


def _plain(t: Optional[torch.Tensor], shape, dtype, device, name: str) -> Optional[int]:
    """Checks a contiguous tensor; its pointer (None for None)."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on {device}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _walkable(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t, or a contiguous copy where no single stride walks its rows."""
    return t if t is None or _stride(t) is not None else t.contiguous()


def _sequences(b: torch.Tensor, seq_off: Optional[torch.Tensor]):
    """(tokens, channels, sequences, offsets pointer) of rows b."""
    if b.dim() == 3:
        if seq_off is not None:
            raise ValueError("seq_off goes with packed [tokens, channels] rows")
        return b.shape[0] * b.shape[1], b.shape[2], b.shape[0], None
    if b.dim() != 2:
        raise ValueError("rows must be [tokens, channels] or [batch, tokens, channels]")
    if seq_off is None:
        return b.shape[0], b.shape[1], 1, None
    if (seq_off.dtype != torch.int32 or seq_off.dim() != 1 or seq_off.numel() < 1 or seq_off.device != b.device
            or not seq_off.is_contiguous()):
        raise ValueError("seq_off must be a contiguous int32 vector on the rows' device")
    return b.shape[0], b.shape[1], seq_off.numel() - 1, seq_off.data_ptr()


@functools.lru_cache(maxsize=256)
def _recur_work(code: int, tokens: int, channels: int) -> int:
    return _lib.load().sla_recur_workspace_bytes(code, tokens, channels)


@functools.lru_cache(maxsize=256)
def _route_work(tokens: int, top_k: int, experts: int) -> int:
    return _lib.load().sla_route_workspace_bytes(tokens, top_k, experts)


def _scratch(size: int, device: torch.device):
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


# ------------------------------------------------------------------------------ recurrence

@_placed
def sla_recur_solve(a: torch.Tensor, b: torch.Tensor, h0: Optional[torch.Tensor] = None,
                    seq_off: Optional[torch.Tensor] = None, *, gate: str = "value",
                    out: Optional[torch.Tensor] = None, h_last: Optional[torch.Tensor] = None):
    """h_t = a_t h_{t-1} + w_t b_t over every sequence; returns (h, last states).

    a, b: [tokens, channels] packed rows, sequence s owning rows seq_off[s] to seq_off[s + 1] (int32,
    on the device; None: one sequence), or [batch, tokens, channels] sequences of one length.
    gate: what a holds ("value": a itself; "exp": its logarithm; "sigmoid": a = sigmoid, and the
    input is weighted by 1 - a).  h0: [sequences, channels] first states (None: zero).  Rows in no
    sequence come back as zeros, or, with `out` given, as they were."""
    code, g = _code(b), _gate(gate)
    tokens, channels, seqs, off = _sequences(b, seq_off)
    lda, ldb = _rows(a, b, "a"), _rows(b, b, "b")
    wide, device = _wide(b.dtype), b.device
    p0 = _plain(h0, (seqs, channels), wide, device, "h0")
    flags = 0
    if out is None:
        out, ldh, flags = torch.empty(b.shape, dtype=b.dtype, device=device), channels, _lib.SLA_FILL_REST
    else:
        ldh = _rows(out, b, "out", out=True)
    if h_last is None:
        h_last = torch.empty((seqs, channels), dtype=wide, device=device)
    size = _recur_work(code, tokens, channels)
    work = _scratch(size, device)
    _check(_lib.load().sla_recur_solve(
        code, g, tokens, channels, seqs, off, a.data_ptr(), lda, b.data_ptr(), ldb, p0, out.data_ptr(), ldh,
        _plain(h_last, (seqs, channels), wide, device, "h_last"), flags,
        None if work is None else work.data_ptr(), size, _current(device)), "sla_recur_solve")
    return out, h_last


@_placed
def sla_recur_adjoint(a: torch.Tensor, h: torch.Tensor, dh: Optional[torch.Tensor], *,
                      b: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                      seq_off: Optional[torch.Tensor] = None, dh_last: Optional[torch.Tensor] = None,
                      gate: str = "value", want_da: bool = True, want_db: bool = True,
                      da: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None):
    """Adjoint of sla_recur_solve: (dL/da, dL/db, dL/dh0) from dh = dL/dh and dh_last = dL/d(last
    states), either of them None for zero.  h: the rows the solve returned; a, h0, seq_off, gate: as
    there; b: its inputs, which the sigmoid gate's dL/da needs.  dL/da is with respect to what a
    holds.  Skipped gradients (want_da, want_db; dL/dh0 without h0) are None; rows in no sequence
    have zero gradients (with `da`, `db` given they stay as they were)."""
    code, g = _code(h), _gate(gate)
    tokens, channels, seqs, off = _sequences(h, seq_off)
    lda, ldh = _rows(a, h, "a"), _rows(h, h, "h")
    wide, device = _wide(h.dtype), h.device
    if gate == "sigmoid" and want_da:
        if b is None:
            raise ValueError("the sigmoid gate's gradient needs b")
        pb, ldb = b, _rows(b, h, "b")
    else:
        pb, ldb = None, 0
    lddh = 0 if dh is None else _rows(dh, h, "dh")
    p0 = _plain(h0, (seqs, channels), wide, device, "h0")
    plast = _plain(dh_last, (seqs, channels), wide, device, "dh_last")
    flags = 0
    if da is None and db is None:
        flags = _lib.SLA_FILL_REST
        da = torch.empty(h.shape, dtype=h.dtype, device=device) if want_da else None
        db = torch.empty(h.shape, dtype=h.dtype, device=device) if want_db else None
    elif (want_da and da is None) or (want_db and db is None):
        raise ValueError("give both da and db, or neither")
    ldda = _rows(da, h, "da", out=True) if want_da else 0
    lddb = _rows(db, h, "db", out=True) if want_db else 0
    dh0 = None if h0 is None else torch.empty((seqs, channels), dtype=wide, device=device)
    size = _recur_work(code, tokens, channels)
    work = _scratch(size, device)
    _check(_lib.load().sla_recur_adjoint(
        code, g, tokens, channels, seqs, off, a.data_ptr(), lda, None if pb is None else pb.data_ptr(), ldb,
        h.data_ptr(), ldh, p0, None if dh is None else dh.data_ptr(), lddh, plast,
        da.data_ptr() if want_da else None, ldda, db.data_ptr() if want_db else None, lddb,
        None if dh0 is None else dh0.data_ptr(), flags,
        None if work is None else work.data_ptr(), size, _current(device)), "sla_recur_adjoint")
    return (da if want_da else None), (db if want_db else None), dh0


@_placed
def sla_recur_step(a: torch.Tensor, b: torch.Tensor, state: torch.Tensor, index: Optional[torch.Tensor] = None, *,
                   gate: str = "value", out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each row of a serving batch: state[index[r]] = a_r state[index[r]] + w_r b_r in
    place; returns the new states' rows in b's type.  a, b: [rows, channels]; state: [slots,
    channels] float32 (float64); index: int32 [rows], distinct (None: row r has slot r).  Rows whose
    index is outside the pool are padding: no state changes, and they come back as zeros (with
    `out` given, as they were)."""
    code, g = _code(b), _gate(gate)
    if b.dim() != 2:
        raise ValueError("rows must be [rows, channels]")
    rows, channels = b.shape
    lda, ldb, device = _rows(a, b, "a"), _rows(b, b, "b"), b.device
    if (state.dim() != 2 or state.shape[1] != channels or state.dtype != _wide(b.dtype) or state.device != device):
        raise ValueError(f"state must be [slots, {channels}] {_wide(b.dtype)} on {device}, got "
                         f"{tuple(state.shape)} {state.dtype} on {state.device}")
    lds = _rows(state, state, "state", out=True)
    if index is None and state.shape[0] < rows:
        raise ValueError("without index every row needs a slot")
    flags = 0
    if out is None:
        out, ldh, flags = torch.empty((rows, channels), dtype=b.dtype, device=device), channels, _lib.SLA_FILL_REST
    else:
        ldh = _rows(out, b, "out", out=True)
    _check(_lib.load().sla_recur_step(
        code, g, rows, channels, state.shape[0], a.data_ptr(), lda, b.data_ptr(), ldb, state.data_ptr(), lds,
        _plain(index, (rows,), torch.int32, device, "index"), out.data_ptr(), ldh, flags, _current(device)),
        "sla_recur_step")
    return out


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


def _check_route(r: Route, device: torch.device):
    tokens, top_k = r.slot.shape
    experts = r.counts.shape[0]
    _plain(r.slot, (tokens, top_k), torch.int32, device, "route.slot")
    _plain(r.offsets, (experts + 1,), torch.int32, device, "route.offsets")
    _plain(r.counts, (experts,), torch.int32, device, "route.counts")
    return tokens, top_k, experts, r.entry.shape[0]


def _side(t: torch.Tensor, rows: int, name: str) -> int:
    """Checks [rows, channels] rows; their row stride."""
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {tuple(t.shape)}")
    return _rows(t, t, name)


@_placed
def sla_route_sort(expert: torch.Tensor, n_experts: int, *, align: int = 1, n_slots: Optional[int] = None) -> Route:
    """The plan that sorts tokens by expert.  expert: [tokens, top_k] (or [tokens]) int32 or int64 ids;
    ids outside [0, n_experts) are dropped.  Within an expert the order is that of the tokens (and
    choices).  Every expert's slots are padded to a multiple of `align` (a product's tile).
    n_slots: slots to provide (default, and least: tokens * top_k + n_experts * (align - 1))."""
    if expert.dtype not in (torch.int32, torch.int64) or expert.dim() not in (1, 2) or not expert.is_contiguous():
        raise ValueError("expert must be a contiguous [tokens, top_k] or [tokens] tensor of int32 or int64")
    device = expert.device
    tokens, top_k = (expert.shape[0], 1) if expert.dim() == 1 else expert.shape
    if n_slots is None:
        n_slots = tokens * top_k + n_experts * (align - 1)
    if n_experts < 1 or align < 1 or top_k < 1 or n_slots < 0 or n_slots >= 2 ** 31:
        raise ValueError("n_experts, align and top_k must be at least 1, and n_slots within [0, 2^31)")
    # one allocation for the plan's four arrays, each on a 16-byte boundary
    up = lambda n: (n + 3) // 4 * 4  # noqa: E731
    o1 = up(n_experts + 1)
    o2 = o1 + up(n_experts)
    o3 = o2 + up(n_slots)
    buf = torch.empty(o3 + tokens * top_k, dtype=torch.int32, device=device)
    route = Route(buf[:n_experts + 1], buf[o1:o1 + n_experts], buf[o2:o2 + n_slots], buf[o3:].view(tokens, top_k))
    size = _route_work(tokens, top_k, n_experts)
    work = _scratch(size, device)
    base = buf.data_ptr()
    _check(_lib.load().sla_route_sort(
        tokens, top_k, n_experts, align, expert.data_ptr(), expert.element_size(), n_slots, base, base + 4 * o1,
        base + 4 * o2, base + 4 * o3, None if work is None else work.data_ptr(), size, _current(device)),
        "sla_route_sort")
    return route


@_placed
def sla_route_dispatch(x: torch.Tensor, route: Route, weight: Optional[torch.Tensor] = None, *,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """xs = R^T x: every slot gets its token's row (times its weight), padding slots zeros.  x:
    [tokens, channels]; weight: [tokens, top_k] float32 (float64) or None for 1.  Slots behind the
    last expert's come back as zeros, or, with `out` given, as they were."""
    return _to_slots(x, route, weight, None, out, False)[0]


@_placed
def sla_route_combine_adjoint(dy: torch.Tensor, route: Route, ys: Optional[torch.Tensor] = None,
                              weight: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None):
    """Adjoint of sla_route_combine: (dL/dys = R^T dy, dL/dweight = dy . ys on R's pattern); the
    latter with ys given, else None.  Dropped entries have weight gradient 0."""
    return _to_slots(dy, route, weight, ys, out, ys is not None)


def _to_slots(x, route, weight, ys, out, want_dw):
    code, device = _code(x), x.device
    tokens, top_k, experts, slots = _check_route(route, device)
    ldx, channels, wide = _side(x, tokens, "rows"), x.shape[1], _wide(x.dtype)
    pw = _plain(weight, (tokens, top_k), wide, device, "weight")
    flags = 0
    if out is None:
        out, ldo, flags = torch.empty((slots, channels), dtype=x.dtype, device=device), channels, _lib.SLA_FILL_REST
    else:
        if out.shape != (slots, channels) or out.dtype != x.dtype or out.device != device:
            raise ValueError(f"out must be {(slots, channels)} {x.dtype} on {device}")
        ldo = _rows(out, out, "out", out=True)
    if not want_dw:
        _check(_lib.load().sla_route_dispatch(
            code, tokens, top_k, experts, slots, channels, x.data_ptr(), ldx, route.offsets.data_ptr(),
            route.counts.data_ptr(), route.slot.data_ptr(), pw, out.data_ptr(), ldo, flags, _current(device)),
            "sla_route_dispatch")
        return out, None
    if ys.shape != (slots, channels) or ys.dtype != x.dtype or ys.device != device:
        raise ValueError(f"ys must be {(slots, channels)} {x.dtype} on {device}")
    ldys = _rows(ys, ys, "ys")
    dw = torch.empty((tokens, top_k), dtype=wide, device=device)
    _check(_lib.load().sla_route_combine_adjoint(
        code, tokens, top_k, experts, slots, channels, x.data_ptr(), ldx, route.offsets.data_ptr(),
        route.counts.data_ptr(), route.slot.data_ptr(), pw, ys.data_ptr(), ldys, out.data_ptr(), ldo, dw.data_ptr(),
        flags, _current(device)), "sla_route_combine_adjoint")
    return out, dw


@_placed
def sla_route_combine(ys: torch.Tensor, route: Route, weight: Optional[torch.Tensor] = None, *,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = R ys: every token's sum over its slots, times their weights ([tokens, top_k] float32 or
    float64; None: 1), in the order of the choices; a token without slots gets zeros.
    ys: [slots, channels]; rows of slots without an entry are not read."""
    return _to_tokens(ys, route, weight, None, out)[0]


@_placed
def sla_route_dispatch_adjoint(dxs: torch.Tensor, route: Route, x: Optional[torch.Tensor] = None,
                               weight: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None):
    """Adjoint of sla_route_dispatch: (dL/dx = R dxs, dL/dweight = x . dxs on R's pattern); the
    latter with x given, else None.  Dropped entries have weight gradient 0."""
    return _to_tokens(dxs, route, weight, x, out)


def _to_tokens(ys, route, weight, x, out):
    code, device = _code(ys), ys.device
    tokens, top_k, _, slots = _check_route(route, device)
    ldys, channels, wide = _side(ys, slots, "rows"), ys.shape[1], _wide(ys.dtype)
    pw = _plain(weight, (tokens, top_k), wide, device, "weight")
    if out is None:
        out, ldo = torch.empty((tokens, channels), dtype=ys.dtype, device=device), channels
    else:
        if out.shape != (tokens, channels) or out.dtype != ys.dtype or out.device != device:
            raise ValueError(f"out must be {(tokens, channels)} {ys.dtype} on {device}")
        ldo = _rows(out, out, "out", out=True)
    if x is None:
        _check(_lib.load().sla_route_combine(
            code, tokens, top_k, slots, channels, ys.data_ptr(), ldys, route.slot.data_ptr(), pw, out.data_ptr(), ldo,
            _current(device)), "sla_route_combine")
        return out, None
    if x.dtype != ys.dtype or x.device != device or x.shape != (tokens, channels):
        raise ValueError(f"x must be {(tokens, channels)} {ys.dtype} on {device}")
    ldx = _rows(x, x, "x")
    dw = torch.empty((tokens, top_k), dtype=wide, device=device)
    _check(_lib.load().sla_route_dispatch_adjoint(
        code, tokens, top_k, slots, channels, ys.data_ptr(), ldys, route.slot.data_ptr(), pw, x.data_ptr(), ldx,
        out.data_ptr(), ldo, dw.data_ptr(), _current(device)), "sla_route_dispatch_adjoint")
    return out, dw


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
