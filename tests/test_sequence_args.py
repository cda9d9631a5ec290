"""Refusals of the sequence operators: argument checks run before any device work, so they are
tested here without a GPU, through the C ABI and the binding's own checks."""
import ctypes as C

import pytest
import torch

import differentiable_sparse_linear_b200 as sla
from differentiable_sparse_linear_b200 import _lib, build, sequence

INVALID, UNSUPPORTED, OK = -1, -5, 0
P = 16   # a pointer that is never followed


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def solve_args(**kw):
    a = dict(dtype=0, gate=0, n_tokens=4, n_chan=8, n_seq=1, off=P, a=P, lda=8, b=P, ldb=8, h0=None, h=P, ldh=8,
             last=None, flags=0, work=None, bytes=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


def adjoint_args(**kw):
    a = dict(dtype=0, gate=0, n_tokens=4, n_chan=8, n_seq=1, off=P, a=P, lda=8, b=None, ldb=0, h=P, ldh=8, h0=None,
             dh=P, lddh=8, dlast=None, dz=P, lddz=8, db=P, lddb=8, dh0=None, flags=0, work=None, bytes=1 << 40,
             stream=None)
    a.update(kw)
    return list(a.values())


def step_args(**kw):
    a = dict(dtype=0, gate=0, n_rows=4, n_chan=8, n_slots=4, a=P, lda=8, b=P, ldb=8, state=P, lds=8, index=None, h=P,
             ldh=8, flags=0, stream=None)
    a.update(kw)
    return list(a.values())


BAD_ROWS = [dict(dtype=4), dict(dtype=-1), dict(gate=3), dict(gate=-1), dict(n_chan=-1), dict(n_chan=2 ** 31),
            dict(flags=2), dict(a=None), dict(lda=7)]


@pytest.mark.parametrize("bad", BAD_ROWS + [
    dict(n_tokens=-1), dict(n_tokens=2 ** 31), dict(n_seq=-1), dict(off=None, n_seq=3), dict(off=None, n_seq=0),
    dict(b=None), dict(ldb=7), dict(h=None), dict(ldh=7), dict(ldh=0), dict(lda=-8)])
def test_solve_refuses(lib, bad):
    assert lib.sla_recur_solve(*solve_args(**bad)) == INVALID
    assert lib.sla_last_error()


@pytest.mark.parametrize("bad", BAD_ROWS + [
    dict(n_tokens=-1), dict(n_seq=-1), dict(h=None), dict(ldh=7), dict(lddh=7), dict(lddz=7), dict(lddz=0),
    dict(lddb=7), dict(gate=2), dict(gate=2, b=P, ldb=3), dict(dh0=P)])
def test_adjoint_refuses(lib, bad):
    assert lib.sla_recur_adjoint(*adjoint_args(**bad)) == INVALID


@pytest.mark.parametrize("bad", BAD_ROWS + [
    dict(n_rows=-1), dict(n_slots=-1), dict(n_slots=2 ** 31), dict(b=None), dict(state=None), dict(lds=7), dict(lds=0),
    dict(h=None), dict(ldh=0)])
def test_step_refuses(lib, bad):
    assert lib.sla_recur_step(*step_args(**bad)) == INVALID


def test_workspace_is_asked_for(lib):
    """A call whose workspace is missing or too small is refused."""
    need = lib.sla_recur_workspace_bytes(0, 100000, 64)
    if need:
        assert lib.sla_recur_solve(*solve_args(n_tokens=100000, n_chan=64, lda=64, ldb=64, ldh=64,
                                               work=P, bytes=need - 1)) == INVALID
        assert lib.sla_recur_solve(*solve_args(n_tokens=100000, n_chan=64, lda=64, ldb=64, ldh=64,
                                               work=None, bytes=need)) == INVALID
    need = lib.sla_route_workspace_bytes(100000, 8, 256)
    if need:
        a = [100000, 8, 256, 1, P, 4, 800000, P, P, P, P]
        assert lib.sla_route_sort(*a, P, need - 1, None) == INVALID
        assert lib.sla_route_sort(*a, None, need, None) == INVALID


def test_empty_problems_need_no_device(lib):
    assert lib.sla_recur_solve(*solve_args(n_chan=0)) == OK
    assert lib.sla_recur_solve(*solve_args(n_tokens=0, n_seq=0)) == OK
    assert lib.sla_recur_adjoint(*adjoint_args(n_chan=0)) == OK
    assert lib.sla_recur_step(*step_args(n_rows=0)) == OK
    assert lib.sla_route_combine(0, 0, 2, 0, 8, None, 8, None, None, None, 8, None) == OK


def sort_args(**kw):
    a = dict(n_tokens=4, top_k=2, n_experts=3, align=1, ids=P, id_bytes=4, n_slots=8, off=P, counts=P, entry=P, slot=P,
             work=P, bytes=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(n_tokens=-1), INVALID), (dict(top_k=0), INVALID), (dict(n_tokens=2 ** 30), INVALID),
    (dict(n_experts=0), INVALID), (dict(n_experts=4097, n_slots=1 << 20), UNSUPPORTED), (dict(align=0), INVALID),
    (dict(id_bytes=2), INVALID), (dict(n_slots=7), INVALID), (dict(align=2, n_slots=10), INVALID),
    (dict(n_slots=2 ** 31), INVALID), (dict(ids=None), INVALID), (dict(off=None), INVALID), (dict(counts=None), INVALID),
    (dict(entry=None), INVALID), (dict(slot=None), INVALID)])
def test_sort_refuses(lib, bad, status):
    assert lib.sla_route_sort(*sort_args(**bad)) == status


def to_slots_args(**kw):
    a = dict(dtype=0, n_tokens=4, top_k=2, n_experts=3, n_slots=8, n_chan=8, x=P, ldx=8, off=P, counts=P, slot=P,
             weight=None, xs=P, ldxs=8, flags=0, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=4), dict(n_tokens=-1), dict(top_k=0), dict(n_tokens=2 ** 31), dict(n_experts=0), dict(n_slots=-1),
    dict(n_chan=-1), dict(x=None), dict(ldx=7), dict(off=None), dict(counts=None), dict(slot=None), dict(xs=None),
    dict(ldxs=7), dict(ldxs=0), dict(flags=4)])
def test_dispatch_refuses(lib, bad):
    assert lib.sla_route_dispatch(*to_slots_args(**bad)) == INVALID


@pytest.mark.parametrize("at,value", [(0, 9), (1, -1), (2, 0), (3, -2), (4, -1), (5, None), (6, 3), (7, None), (9, None),
                                      (10, 0)])
def test_combine_refuses(lib, at, value):
    a = [0, 4, 2, 8, 8, P, 8, P, None, P, 8, None]
    a[at] = value
    assert lib.sla_route_combine(*a) == INVALID


def test_adjoints_of_routing_refuse(lib):
    good = [0, 4, 2, 8, 8, P, 8, P, None, P, 8, P, 8, P, None]
    for at, value in ((0, 7), (5, None), (9, None), (10, 5), (11, None), (12, 2)):
        a = list(good)
        a[at] = value
        assert lib.sla_route_dispatch_adjoint(*a) == INVALID, at
    good = [0, 4, 2, 3, 8, 8, P, 8, P, P, P, None, P, 8, P, 8, P, 0, None]
    for at, value in ((0, 7), (3, 0), (6, None), (8, None), (9, None), (10, None), (12, None), (13, 2), (14, None),
                      (15, 0), (17, 8)):
        a = list(good)
        a[at] = value
        assert lib.sla_route_combine_adjoint(*a) == INVALID, at


# ------------------------------------------------------------------------- the binding's checks

def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 8)
    off = torch.tensor([0, 4], dtype=torch.int32)
    route = sla.Route(off, off[:1], off, torch.zeros(4, 1, dtype=torch.int32))
    for call in (lambda: sla.sla_recur_solve(x, x), lambda: sla.recurrence(x, x), lambda: sla.sla_recur_adjoint(x, x, x),
                 lambda: sla.sla_recur_step(x, x, x), lambda: sla.sla_route_sort(off, 3),
                 lambda: sla.sla_route_dispatch(x, route), lambda: sla.sla_route_combine(x, route),
                 lambda: sla.route_dispatch(x, route), lambda: sla.route_combine(x, route),
                 lambda: sla.sla_recur_solve(a=x, b=x), lambda: sla.sla_recur_solve([1.0], [2.0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_row_strides():
    s = sequence._stride
    x = torch.zeros(6, 8)
    assert s(x) == 8 and s(x[:, :5]) == 8 and s(x[::2]) == 16
    assert s(x[:1].expand(6, 8)) == 0                      # one row for all
    assert s(x.t()) is None                                # channels apart
    assert s(x[:, ::2]) is None
    assert s(torch.zeros(8).as_strided((4, 4), (1, 1))) is None   # rows overlap
    y = torch.zeros(2, 3, 8)
    assert s(y) == 8 and s(y.transpose(0, 1)) is None and s(y[:, :2]) is None and s(y[:1, :2]) == 8
    assert s(torch.zeros(5, 3, 8)[:, :1]) == 24            # one row a sequence
    assert s(torch.zeros(8).expand(2, 3, 8)) == 0
    assert s(torch.zeros(1, 8)) == 8 and s(torch.zeros(0, 8)) == 8
    assert s(torch.zeros(6, 2)[:, :1]) == 2
    assert s(sequence._walkable(y.transpose(0, 1))) == 8


def test_binding_refuses():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="overlap"):
        sequence._rows(x[:1].expand(4, 8), x, "out", out=True)
    with pytest.raises(ValueError, match="stride"):
        sequence._rows(x.t(), x.t(), "a")
    with pytest.raises(ValueError, match="must be"):
        sequence._rows(x.double(), x, "a")
    with pytest.raises(ValueError, match="must be"):
        sequence._rows(x[:3], x, "a")
    with pytest.raises(ValueError, match="contiguous"):
        sequence._plain(x.t(), (8, 4), torch.float32, x.device, "h0")
    with pytest.raises(ValueError, match="must be"):
        sequence._plain(x, (8, 4), torch.float32, x.device, "h0")
    with pytest.raises(ValueError, match="rows must be"):
        sequence._code(x.to(torch.int32))
    with pytest.raises(ValueError, match="gate"):
        sequence._gate("tanh")
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="packed"):
        sequence._sequences(x[None], off)
    for bad in (off.long(), off[:0], off[None], torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="seq_off"):
            sequence._sequences(x, bad)
    with pytest.raises(ValueError, match="rows must be"):
        sequence._sequences(x[0], None)
