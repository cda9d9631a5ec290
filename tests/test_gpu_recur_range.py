"""The recurrence where numbers leave their range or are not finite: its results are those of the row-by-row
form, wherever a sequence lies in the packed rows (tiles are 176 rows long forward, 160 or 144 backward)."""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_b200 as sla
import sequence_reference as ref

pytestmark = pytest.mark.gpu


def by_rows(a, b, h0, off, gate):
    """The definition in 64 bits: every coefficient is used, the first one of a sequence on 0 without h0."""
    h, last = np.zeros(b.shape), np.zeros((len(off) - 1, b.shape[1]))
    with np.errstate(all="ignore"):
        for s in range(len(off) - 1):
            v = np.zeros(b.shape[1]) if h0 is None else h0[s]
            for t in range(off[s], off[s + 1]):
                c, w = ref.gate_of(a[t], gate)
                v = c * v + w * b[t]
                h[t] = v
            last[s] = v
    return h, last


def same_where_finite(got, want, bound):
    got = ref.host(got)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), np.argwhere(np.isfinite(got) != np.isfinite(want))[:4]
    ok = np.isfinite(want)
    assert (np.abs(got - np.where(ok, want, 0))[ok] <= bound[ok]).all()


STARTS = [0, 1, 3, 4, 143, 144, 145, 159, 160, 161, 175, 176, 177, 300]
BEYOND = {"value": [np.nan, np.inf, -np.inf], "exp": [np.nan, np.inf], "sigmoid": [np.nan]}


@pytest.mark.parametrize("gate,kind", [("value", "f32"), ("value", "f64"), ("value", "f16"), ("exp", "bf16"),
                                       ("exp", "f32"), ("sigmoid", "bf16"), ("sigmoid", "f64")])
@pytest.mark.parametrize("first", [True, False])
def test_coefficients_that_are_not_finite(gate, kind, first):
    """One such coefficient a channel: at the sequence's first row, inside a run of four rows, at and around tiles' ends;
    over zero rows and zero states and over others."""
    kind, n = ref.KINDS[kind], 430
    at = [0, 1, 2, 3, 4, 7, 143, 144, 159, 160, 175, 176, 177, 320, 429]
    cases = [(j, v, zeros) for j in at for v in BEYOND[gate] for zeros in (False, True)]
    d = len(cases)
    g = torch.Generator().manual_seed(7)
    z = torch.randn(n, d, generator=g) + 1
    a = {"value": torch.sigmoid(z), "exp": torch.nn.functional.logsigmoid(z), "sigmoid": z}[gate]
    b, h0 = torch.randn(n, d, generator=g), torch.randn(1, d, generator=g)
    dh, dlast = torch.randn(n, d, generator=g), torch.randn(1, d, generator=g)
    for c, (j, v, zeros) in enumerate(cases):
        a[j, c] = v
        if zeros:                                          # nothing in front of it, in either direction
            b[:j + 1, c] = h0[0, c] = 0
            dh[j:, c] = dlast[0, c] = 0
    masks = None
    for s in STARTS:
        rows = lambda t: torch.cat([torch.full((s, d), 0.5), t, torch.full((20, d), 0.5)]).to(kind).cuda()  # noqa: E731
        A, B, D = rows(a), rows(b), rows(dh)
        off = [0, s, s + n, s + n + 20]
        o = torch.tensor(off, dtype=torch.int32).cuda()
        few = lambda t: torch.cat([torch.ones(1, d), t, torch.ones(1, d)]).to(ref.wide(kind)).cuda()  # noqa: E731
        first0, dl = few(h0) if first else None, few(dlast)
        h, last = sla.sla_recur_solve(A, B, first0, o, gate=gate)
        want, wlast = by_rows(ref.host(A), ref.host(B), None if first0 is None else ref.host(first0), off, gate)
        with np.errstate(all="ignore"):
            _, _, e, elast = ref.solve(ref.host(A), ref.host(B), None if first0 is None else ref.host(first0), off, gate, kind)
            # the rows in front are another sequence, only there to move this one (exp: they grow out of fp32's range)
            same_where_finite(h[s:], want[s:], ref.storage(want, e, kind)[s:])
            same_where_finite(last[1:], wlast[1:], ref.storage(wlast, elast, ref.wide(kind))[1:])
            back = sla.sla_recur_adjoint(A, B, D, b=B, h0=first0, seq_off=o, dh_last=dl, gate=gate)   # B: any finite rows
            wants = ref.adjoint(ref.host(A), ref.host(B), ref.host(B), None if first0 is None else ref.host(first0),
                                ref.host(D), ref.host(dl), off, gate, kind)
            for name, t in zip(("da", "db", "dh0"), back):
                if t is not None:
                    w, e = wants[name]
                    bound, k = ref.storage(w, e, ref.wide(kind) if name == "dh0" else kind), 1 if name == "dh0" else s
                    same_where_finite(t[k:], w[k:], bound[k:])
        mask = torch.cat([torch.isfinite(t[s:s + n]) for t in (h, back[0], back[1])])
        masks = mask if masks is None else masks
        assert torch.equal(mask, masks)
