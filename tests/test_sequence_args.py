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
# Shapes, types and strides are looked at before the device, so host tensors reach every refusal.

@pytest.fixture(scope="module")
def native(lib):
    return sequence._load()


def plan(tokens=4, top_k=1, experts=1, slots=4):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return sla.Route(z(experts + 1), z(experts), z(slots), z(tokens, top_k))


def test_cpu_tensors_are_refused(native):
    x, s = torch.zeros(4, 8), torch.zeros(1, 8)
    ids = torch.zeros(4, dtype=torch.int32)
    route = plan()
    for call in (lambda: sla.sla_recur_solve(x, x), lambda: sla.recurrence(x, x), lambda: sla.sla_recur_adjoint(x, x, x),
                 lambda: sla.sla_recur_step(x, x, x.clone()), lambda: sla.sla_route_sort(ids, 3),
                 lambda: sla.sla_route_dispatch(x, route), lambda: sla.sla_route_combine(x, route),
                 lambda: sla.route_dispatch(x, route), lambda: sla.route_combine(x, route),
                 lambda: sla.sla_recur_solve(a=x, b=x, h0=s), lambda: sla.sla_recur_solve([1.0], [2.0]),
                 lambda: sla.sla_recur_solve(x, None), lambda: sla.sla_recur_solve(x, x, stream=0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_row_strides(native):
    s = native.stride_of
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


def test_shared_memory(native):
    shared = native.share_memory
    x = torch.zeros(7, 12)
    cases = [(x, x, True), (x[:4], x[4:], False), (x[:4], x[3:], True), (x[::2], x[1::2], False),
             (x[:, :4], x[:, 4:], False), (x[:, 4:], x[:, :4], False), (x[:, :5], x[:, 4:], True),
             (x[1:, :4], x[:-1, 4:], False), (x[1:, :5], x[:-1, 4:], True), (x[:, 8:], x[2:3, :8], False),
             (x[:, 8:], x[2:3, :9], True), (x[2:3, :9], x[:, 8:], True), (x[:1, :3], x[:1, 3:], False),
             (x[:1, :4], x[:1, 3:], True), (x[3:4].expand(5, 12), x[:4], True), (x[3:4].expand(5, 12), x[:3], False),
             (x[:, :4], torch.zeros(7, 12), False), (x[::2], x[:, :4], True), (x[:0], x, False),
             (x.view(-1)[:36].view(3, 12), x.view(-1)[30:66].view(3, 12), True)]
    for p, q, expected in cases:
        assert shared(p, q) is expected and shared(q, p) is expected
        cells = [set((t.storage_offset() + (torch.arange(t.shape[0])[:, None] * t.stride(0) +
                                            torch.arange(t.shape[1]) * t.stride(1))).flatten().tolist()) for t in (p, q)]
        same = p.untyped_storage().data_ptr() == q.untyped_storage().data_ptr()
        meet = same and bool(cells[0] & cells[1])
        assert expected or not meet                        # what shares memory is never missed


def test_shifted_rows_are_refused(native):
    x = torch.zeros(9, 8)
    y = torch.zeros(8, 8)
    for call in (lambda: sla.sla_recur_solve(y, x[:-1], out=x[1:]),
                 lambda: sla.sla_recur_solve(x[1:], y, out=x[:-1]),
                 lambda: sla.sla_recur_adjoint(y, y, x[1:], da=x[:-1], db=y.clone()),
                 lambda: sla.sla_recur_adjoint(y, y, y, da=x[1:], db=x[:-1]),
                 lambda: sla.sla_recur_step(y, x[1:], x[:-1]),
                 lambda: sla.sla_recur_solve(y, y, x[:1], out=x[:8])):
        with pytest.raises(ValueError, match="other arguments"):
            call()
    wide = torch.zeros(8, 16)                              # columns of one buffer are not: these fail as CPU tensors
    with pytest.raises(ValueError, match="CUDA"):
        sla.sla_recur_solve(wide[:, :8], y, out=wide[:, 8:])


def test_recurrence_refuses(native):
    x, y = torch.zeros(4, 8), torch.zeros(4, 8)
    off = torch.tensor([0, 4], dtype=torch.int32)
    solve, adjoint, step = sla.sla_recur_solve, sla.sla_recur_adjoint, sla.sla_recur_step
    for call, words in [
            (lambda: solve(x, x, out=x[:1].expand(4, 8)), "overlap"),
            (lambda: solve(x.t(), x.t()), "stride"),
            (lambda: solve(x.double(), x), "a must be"),
            (lambda: solve(x[:3], x), "a must be"),
            (lambda: solve(x, x, out=x.bfloat16()), "out must be"),
            (lambda: solve(x, x, torch.zeros(8, 1).t()[:, ::2], off), "h0 must be"),
            (lambda: solve(x, x, torch.zeros(2, 8), off), "h0 must be"),
            (lambda: solve(x, x, torch.zeros(1, 8).double(), off), "h0 must be"),
            (lambda: solve(x[:, :1], x[:, :1], torch.zeros(2, 2)[:, :1], torch.zeros(3, dtype=torch.int32)), "contiguous"),
            (lambda: solve(x, x, h_last=torch.zeros(2, 8)), "h_last must be"),
            (lambda: solve(x.int(), x.int()), "rows must be"),
            (lambda: solve(x, x, gate="tanh"), "gate"),
            (lambda: solve(x, x, gate=None), "gate"),
            (lambda: solve(x[None], x[None], None, off), "packed"),
            (lambda: solve(x[0], x[0]), "rows must be"),
            (lambda: adjoint(x, x, x, gate="sigmoid"), "needs b"),
            (lambda: adjoint(x, x, x, da=x.clone()), "both"),
            (lambda: adjoint(x, x, x[:2]), "dh must be"),
            (lambda: adjoint(x, x, x, dh_last=torch.zeros(3, 8)), "dh_last must be"),
            (lambda: adjoint(x, x, x, da=x[:1].expand(4, 8), db=x.clone()), "overlap"),
            (lambda: adjoint(x, x, x, b=x[:, ::2], gate="sigmoid"), "b must be"),
            (lambda: step(x, x, x[:3]), "slot"),
            (lambda: step(x, x, x.bfloat16()), "state must be"),
            (lambda: step(x, x, x[:1].expand(4, 8)), "overlap"),
            (lambda: step(x, x, y, torch.arange(4)), "index must be"),
            (lambda: step(x, x, y, torch.zeros(3, dtype=torch.int32)), "index must be"),
            (lambda: step(x[None], x[None], x), "rows must be"),
            (lambda: solve(x, y, out=y), "other arguments"),
            (lambda: solve(x, y, torch.zeros(1, 8), h_last=x[:1]), "other arguments"),
            (lambda: adjoint(x, y, y, da=y, db=x.clone()), "other arguments"),
            (lambda: step(x, y, x), "other arguments")]:
        with pytest.raises(ValueError, match=words):
            call()
    for bad in (off.long(), off[:0], off[None], torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="seq_off"):
            solve(x, x, None, bad)


def test_routing_refuses(native):
    x, w = torch.zeros(4, 8), torch.zeros(4, 1)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    r = plan()
    for call, words in [
            (lambda: sla.sla_route_sort(ids.float(), 3), "expert must be"),
            (lambda: sla.sla_route_sort(ids[:, :1], 3), "expert must be"),
            (lambda: sla.sla_route_sort(ids[None], 3), "expert must be"),
            (lambda: sla.sla_route_sort(ids, 0), "at least 1"),
            (lambda: sla.sla_route_sort(ids, 3, align=0), "at least 1"),
            (lambda: sla.sla_route_sort(ids[:, :0].contiguous(), 3), "at least 1"),
            (lambda: sla.sla_route_sort(ids, 3, align=2 ** 30), "n_slots"),
            (lambda: sla.sla_route_sort(ids, 3, n_slots=-1), "n_slots"),
            (lambda: sla.sla_route_sort(ids, 2.5), "whole"),
            (lambda: sla.sla_route_dispatch(x[:3], r), "rows must be"),
            (lambda: sla.sla_route_dispatch(x.int(), r), "rows must be"),
            (lambda: sla.sla_route_dispatch(x.t(), plan(tokens=8)), "stride"),
            (lambda: sla.sla_route_dispatch(x, r, w.double()), "weight must be"),
            (lambda: sla.sla_route_dispatch(x, r, w[:, 0]), "weight must be"),
            (lambda: sla.sla_route_dispatch(x, r, out=x), "other arguments"),
            (lambda: sla.sla_route_combine(x, r, out=x), "other arguments"),
            (lambda: sla.sla_route_dispatch(x, r, out=x[:3]), "out must be"),
            (lambda: sla.sla_route_dispatch(x, r, out=x[:1].expand(4, 8)), "overlap"),
            (lambda: sla.sla_route_dispatch(x, sla.Route(r.offsets, r.counts, r.entry, r.slot.long())), "route.slot"),
            (lambda: sla.sla_route_dispatch(x, sla.Route(r.counts, r.counts, r.entry, r.slot)), "route.offsets"),
            (lambda: sla.sla_route_combine(x, plan(slots=5)), "rows must be"),
            (lambda: sla.sla_route_combine(x, r, out=x.double()), "out must be"),
            (lambda: sla.sla_route_dispatch_adjoint(x, r, x[:, :4]), "x must be"),
            (lambda: sla.sla_route_combine_adjoint(x, r, x.bfloat16()), "ys must be")]:
        with pytest.raises(ValueError, match=words):
            call()


def test_workspace_sizes(lib):
    """A call of several tiles or blocks needs a workspace, and says so; one of a single tile does not."""
    rows = dict(n_tokens=100000, n_chan=64, lda=64, ldb=64, ldh=64)
    for dtype, width in ((0, 4), (1, 8), (2, 4), (3, 4)):
        need = lib.sla_recur_workspace_bytes(dtype, 100000, 64)
        assert need >= 100000 // 176 * 64 * 3 * width        # a map and a state a channel of every tile
        assert lib.sla_recur_solve(*solve_args(dtype=dtype, work=P, bytes=need - 1, **rows)) == INVALID
        assert lib.sla_recur_solve(*solve_args(dtype=dtype, work=None, bytes=need, **rows)) == INVALID
        assert lib.sla_recur_solve(*solve_args(dtype=dtype, work=P + 8, bytes=need, **rows)) == INVALID
        assert lib.sla_recur_workspace_bytes(dtype, 144, 64) == 0
    need = lib.sla_route_workspace_bytes(100000, 8, 256)
    assert need >= 2 * 256 * 4                             # a histogram a block
    a = [100000, 8, 256, 1, P, 4, 800000, P, P, P, P]
    assert lib.sla_route_sort(*a, P, need - 1, None) == INVALID
    assert lib.sla_route_sort(*a, None, need, None) == INVALID
    assert lib.sla_route_workspace_bytes(1000, 8, 256) == 0
