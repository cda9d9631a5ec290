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


def overshoots(kind):
    """({row: exponent of a}, {row: exponent of b}, exponent of the first state, sign) of columns whose states stay in
    range while products of coefficients, or sums from a zero state, overflow.  Powers of two: every state is exact.
    No two neighbouring coefficients have a product below 2^-126 (fp64 2^-1022), which may count as 0."""
    s = 8 if kind == torch.float64 else 1
    top = 1023 if s == 8 else 127
    out = []
    for p in (0, 1, 3, 5, 100, 160, 172, 175, 176, 177, 300):
        for sign in (1, -1):
            for a, first in (({p: 50, p + 4: 50, p + 16: 66, p + 20: -66}, -100), ({p + 12: 100, p + 16: 66, p + 20: -66}, -83),
                             ({p: 100, p + 1: 100, p + 2: -50, p + 3: -50}, -80), ({p: 70, p + 176: 70, p + 352: -70}, -100),
                             ({p: 100, p + 40: 100}, -120), ({p: 100, p + 3: 60, p + 9: 60, p + 90: -60}, -120)):
                out.append(({r: e * s for r, e in a.items()}, {}, first * s, sign))
        out.append(({}, {p: top, p + 50: top}, top, 0))       # -2^top, then 0, then 2^top
    return out


@pytest.mark.parametrize("kind", ["f32", "f64", "bf16"])
@pytest.mark.parametrize("off", [[0, 800], [3, 783], [0, 200, 200, 790], [0, 5, 170, 185, 800]])
def test_products_beyond_the_range(kind, off):
    """The states are those of the rows one after the other, bit for bit: backward the same columns, reversed."""
    kind = ref.KINDS[kind]
    cases, n = overshoots(kind), len(off) - 1
    T, d = 800, len(cases)
    a, b, first = np.ones((T, d)), np.zeros((T, d)), np.zeros((n, d))
    for c, (ea, eb, e0, sign) in enumerate(cases):
        for s in range(n):                                 # in every sequence, from its first row on
            for r, e in ea.items():
                if off[s] + r < off[s + 1]:
                    a[off[s] + r, c] = (sign if r % 4 == 0 else 1) * 2.0 ** e
            for r, e in eb.items():
                if off[s] + r < off[s + 1]:
                    b[off[s] + r, c] = 2.0 ** e
            first[s, c] = -2.0 ** e0 if sign == 0 else 2.0 ** e0
    put = lambda x, k: torch.from_numpy(x).to(k).cuda()  # noqa: E731
    o = torch.tensor(off, dtype=torch.int32).cuda()
    want, wlast = by_rows(a, b, first, off, "value")
    assert np.isfinite(want).all() and np.abs(want).max() < torch.finfo(kind).max
    for pad in (0, 1):                                     # aligned rows and others
        A, B = (torch.nn.functional.pad(put(x, kind), (0, pad)) for x in (a, b))
        h, last = sla.sla_recur_solve(A[:, :d], B[:, :d], put(first, ref.wide(kind)), o)
        assert np.array_equal(ref.host(h), want) and np.array_equal(ref.host(last), wlast)
        # lambda_t = g_t + a_{t+1} lambda_{t+1}: with a and b turned round, the last state is dL/dh_last and the
        # states (before the coefficient) are those of the reversed rows
        ra, rb, roff = a[::-1].copy(), b[::-1].copy(), [T - v for v in off[::-1]]
        lam, dh0 = np.zeros((T, d)), np.zeros((n, d))
        for s in range(n):
            v = first[::-1][s]
            for t in range(roff[s + 1] - 1, roff[s] - 1, -1):
                lam[t] = rb[t] + v
                v = ra[t] * lam[t]
            dh0[s] = v
        ro = torch.tensor(roff, dtype=torch.int32).cuda()
        RA, RB = (torch.nn.functional.pad(put(x, kind), (0, pad)) for x in (ra, rb))
        ok = np.isfinite(lam).all(0) & (np.abs(lam) < torch.finfo(kind).max).all(0) & (np.abs(dh0) < torch.finfo(kind).max).all(0)
        assert ok.sum() > d // 2
        da, db, got0 = sla.sla_recur_adjoint(RA[:, :d], torch.zeros_like(RA)[:, :d], RB[:, :d], h0=torch.zeros_like(put(first, ref.wide(kind))),
                                             seq_off=ro, dh_last=put(first[::-1].copy(), ref.wide(kind)))
        assert np.array_equal(ref.host(db)[:, ok], lam[:, ok]) and np.array_equal(ref.host(got0)[:, ok], dh0[:, ok])
        assert (ref.host(da)[:, ok] == 0).all()


@pytest.mark.parametrize("back", [False, True])
def test_coefficients_close_to_one_over_many_tiles(back):
    """A state of 1 over a thousand coefficients of 1 - 3 * 2^-24, one a tile, and ones: products and sums are exact
    but for the coefficients' own, u = 2^-24 relative each, and one more where a tile's rows get their states.  Products
    held in fewer than 24 bits lose up to 3 u a tile."""
    rows, n, d, u = (160 if back else 176), 1000, 8, 2.0 ** -24
    c = 1 - 3 * u
    a = torch.ones(n * rows, d)
    at = torch.arange(n) * rows + 5
    a[n * rows - 1 - at if back else at] = c
    zero = torch.zeros(n * rows, d, device="cuda")
    used = np.zeros(n * rows)
    used[at.numpy()] = 1
    k = np.cumsum(used)
    one = torch.ones(1, d, device="cuda")
    if back:
        _, got, end = sla.sla_recur_adjoint(a.cuda(), zero, None, h0=one, dh_last=one)
        got, k = got.flip(0), k - used                     # lambda is in front of its row's coefficient
    else:
        got, end = sla.sla_recur_solve(a.cuda(), zero, one)
    want = np.exp(k * np.log1p(-3 * u))[:, None] * np.ones((1, d))
    ref.within(got, want, (k[:, None] + 2) * u * want)
    ref.within(end, want[-1:], (n + 2) * u * want[-1:])
