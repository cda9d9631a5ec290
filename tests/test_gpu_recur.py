"""Gated linear recurrence on the GPU against the row-by-row 64-bit form: solve, adjoint, step and
their autograd function, at the lengths, strides and packings where they can go wrong.  Bounds are
derived in sequence_reference.py."""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_b200 as sla
import sequence_reference as ref

pytestmark = pytest.mark.gpu

# tokens and offsets: one row, around the lengths a kernel may cut time at, ragged with empty
# sequences, rows in front of the first and behind the last one, single rows, nothing at all
PACKINGS = {
    "one": (1, [0, 1]),
    "two_rows": (2, [0, 2]),
    "short": (37, [0, 37]),
    "cut-1": (255, [0, 255]), "cut": (256, [0, 256]), "cut+1": (257, [0, 257]),
    "cut128": (129, [0, 128, 129]), "cut512": (513, [0, 1, 512, 513]),
    "ragged": (700, [0, 3, 3, 131, 290, 290, 290, 291, 640, 700]),
    "rest": (300, [7, 7, 40, 260, 260]),
    "singles": (70, list(range(71))),
    "empties": (5, [5, 5, 5]),
    "none": (6, [3]),
    "long": (3000, [0, 1999, 2000, 3000]),
}


def data(packing, d, kind, gate, seed=0, first=True):
    tokens, off = PACKINGS[packing] if isinstance(packing, str) else packing
    g = torch.Generator().manual_seed(1000 * seed + tokens * 7 + d)
    z = torch.randn(tokens, d, generator=g) + 2 * torch.rand(d, generator=g)
    a = {"value": torch.sigmoid(z), "exp": torch.nn.functional.logsigmoid(z), "sigmoid": z}[gate]
    if gate == "value":     # some coefficients negative, zero, one and above one
        a[torch.rand(tokens, d, generator=g) < 0.1] *= -1
        a[torch.rand(tokens, d, generator=g) < 0.02] = 0
        a[torch.rand(tokens, d, generator=g) < 0.02] = 1.0
        a[torch.rand(tokens, d, generator=g) < 0.02] = 1.25
    wide = ref.wide(kind)
    n = len(off) - 1
    return dict(off=torch.tensor(off, dtype=torch.int32).cuda(), offsets=off, a=a.to(kind).cuda(),
                b=torch.randn(tokens, d, generator=g).to(kind).cuda(),
                h0=torch.randn(n, d, generator=g).to(wide).cuda() if first else None,
                dh=torch.randn(tokens, d, generator=g).to(kind).cuda(),
                dlast=torch.randn(n, d, generator=g).to(wide).cuda())


def opt(t):
    return None if t is None else ref.host(t)


def check_solve(x, h, last, gate, kind):
    want, wlast, e, elast = ref.solve(ref.host(x["a"]), ref.host(x["b"]), opt(x["h0"]), x["offsets"], gate, kind)
    ref.within(h, want, ref.storage(want, e, kind))
    ref.within(last, wlast, ref.storage(wlast, elast, ref.wide(kind)))
    return want


def check_adjoint(x, h, got, gate, kind, dh=True, dlast=True):
    want = ref.adjoint(ref.host(x["a"]), ref.host(x["b"]), ref.host(h), opt(x["h0"]),
                       ref.host(x["dh"]) if dh else None, ref.host(x["dlast"]) if dlast else None, x["offsets"], gate, kind)
    for name, t in zip(("da", "db", "dh0"), got):
        if t is not None:
            v, e = want[name]
            ref.within(t, v, ref.storage(v, e, ref.wide(kind) if name == "dh0" else kind))


@pytest.mark.parametrize("packing", PACKINGS)
@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("gate", sla.GATES)
def test_solve_and_adjoint(packing, kind, gate):
    kind = ref.KINDS[kind]
    for d, first in ((64, True), (1, False), (33, True), (130, False), (8, True)):
        x = data(packing, d, kind, gate, first=first)
        h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate=gate)
        check_solve(x, h, last, gate, kind)
        got = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"],
                                    gate=gate)
        assert (got[2] is not None) == first
        check_adjoint(x, h, got, gate, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("d", [2, 4, 7, 16, 31, 32, 72, 100, 257, 1000])
def test_widths(kind, d):
    kind = ref.KINDS[kind]
    x = data("ragged", d, kind, "sigmoid")
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="sigmoid")
    check_solve(x, h, last, "sigmoid", kind)
    got = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"],
                                gate="sigmoid")
    check_adjoint(x, h, got, "sigmoid", kind)


@pytest.mark.parametrize("kind,gate", [("f32", "value"), ("bf16", "exp"), ("f64", "sigmoid")])
def test_long_sequence(kind, gate):
    """Many time chunks, few channels, and a sequence border far in."""
    kind = ref.KINDS[kind]
    x = data((40000, [0, 33333, 40000]), 24, kind, gate)
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate=gate)
    check_solve(x, h, last, gate, kind)
    got = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate=gate)
    check_adjoint(x, h, got, gate, kind)


@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("gate", ["exp", "sigmoid"])
@pytest.mark.parametrize("d", [64, 33])
def test_gates_at_their_ends(kind, gate, d):
    """Gates so far out that a coefficient or 1 minus it is 0, infinite ones among them.

    Bound: besides the relative errors, a coefficient or weight below 2^-124 (fp64: 2^-1009) may be anything up to
    that, where the arithmetic holds it or flushes it.  In 300 rows, values below 6 (asserted), |h| and |lambda| stay below
    301 * 6 < 2^11, every product of the two below 2^22, and 300 such errors add up to less than
    2^-124 * 2^22 * 2^9."""
    kind = ref.KINDS[kind]
    ends = [-float("inf"), -6e4, -1000.0, -200.0, -95.0, -88.0, -40.0, -17.0, -1.0, -0.0, 0.0]
    if gate == "sigmoid":
        ends += [-v for v in ends[:-2]]
    x = data((300, [0, 7, 120, 290]), d, kind, gate)
    pick = torch.randint(len(ends), x["a"].shape, generator=torch.Generator().manual_seed(d))
    x["a"] = torch.tensor(ends, dtype=torch.float64)[pick].to(kind).cuda()
    assert all(float(x[k].abs().max()) < 6 for k in ("b", "h0", "dh", "dlast"))
    extra = (2.0 ** -1009 if kind == torch.float64 else 2.0 ** -124) * 2.0 ** 31
    za, zb, zh0 = ref.host(x["a"]), ref.host(x["b"]), ref.host(x["h0"])
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate=gate)
    want, wlast, e, elast = ref.solve(za, zb, zh0, x["offsets"], gate, kind)
    ref.within(h, want, ref.storage(want, e + extra, kind))
    ref.within(last, wlast, ref.storage(wlast, elast + extra, ref.wide(kind)))
    got = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate=gate)
    want = ref.adjoint(za, zb, ref.host(h), zh0, ref.host(x["dh"]), ref.host(x["dlast"]), x["offsets"], gate, kind)
    for name, t in zip(("da", "db", "dh0"), got):
        v, e = want[name]
        ref.within(t, v, ref.storage(v, e + extra, ref.wide(kind) if name == "dh0" else kind))
    state = x["h0"][:1].expand(7, d).contiguous()          # and the single step
    h = sla.sla_recur_step(x["a"][:7], x["b"][:7], state, gate=gate)
    for r in range(7):
        w, _, e, _ = ref.solve(za[r:r + 1], zb[r:r + 1], zh0[:1], [0, 1], gate, kind)
        ref.within(h[r:r + 1], w, ref.storage(w, e + extra, kind))


def test_slow_decay_keeps_far_inputs():
    """Coefficients of 1 sum: an input reaches every later row through all chunks."""
    tokens, d = 5000, 40
    a, b = torch.ones(tokens, d, device="cuda"), torch.zeros(tokens, d, device="cuda")
    b[0], b[777] = 1.0, 2.0
    h, last = sla.sla_recur_solve(a, b)
    want = torch.ones(tokens, d, device="cuda")
    want[777:] = 3
    assert torch.equal(h, want) and torch.equal(last, want[-1:])


def test_growth_and_zero_rows():
    """Coefficients of 2 over zero rows (a product that leaves fp32's range) change nothing; a state that
    leaves the range is infinite, as in the row-by-row form."""
    tokens, d = 1500, 16
    a, b = torch.full((tokens, d), 2.0, device="cuda"), torch.zeros(tokens, d, device="cuda")
    b[1490] = 1.0
    h, _ = sla.sla_recur_solve(a, b)
    want = torch.zeros(tokens, d, device="cuda")
    for t in range(1490, tokens):
        want[t] = 2.0 ** (t - 1490)
    assert torch.equal(h, want)
    b[3] = 1.0
    h, last = sla.sla_recur_solve(a, b)
    assert torch.equal(h[100], torch.full((d,), 2.0 ** 97, device="cuda"))
    assert torch.isinf(h[200:]).all() and torch.isinf(last).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_batch_layouts(kind):
    """[batch, tokens, channels] rows, rows with a stride, one coefficient row for all tokens."""
    kind = ref.KINDS[kind]
    B, T, d = 3, 291, 48
    off = [0, T, 2 * T, 3 * T]
    x = data((B * T, off), d, kind, "value")
    view = lambda t: t.view(B, T, d)  # noqa: E731
    h, last = sla.sla_recur_solve(view(x["a"]), view(x["b"]), x["h0"], gate="value")
    assert h.shape == (B, T, d)
    check_solve(x, h.reshape(-1, d), last, "value", kind)
    got = sla.sla_recur_adjoint(view(x["a"]), h, view(x["dh"]), h0=x["h0"], dh_last=x["dlast"])
    check_adjoint(x, h.reshape(-1, d), (got[0].reshape(-1, d), got[1].reshape(-1, d), got[2]), "value", kind)
    # the two inputs side by side in one buffer, the output in a third column block of it
    for pad in (16, 3):
        buf = torch.full((B * T, 3 * d + pad), 7.0, dtype=kind, device="cuda")
        buf[:, :d], buf[:, d:2 * d] = x["a"], x["b"]
        out = buf[:, 2 * d + pad:]
        h2, last2 = sla.sla_recur_solve(buf[:, :d], buf[:, d:2 * d], x["h0"], x["off"], out=out)
        assert torch.equal(h2.contiguous(), h.reshape(-1, d)) and torch.equal(last2, last)
        assert (buf[:, 2 * d:2 * d + pad] == 7).all()
    one = x["a"][:1].expand(B * T, d)
    h3, last3 = sla.sla_recur_solve(one, x["b"], x["h0"], x["off"])
    h4, last4 = sla.sla_recur_solve(one.contiguous(), x["b"], x["h0"], x["off"])
    assert torch.equal(h3, h4) and torch.equal(last3, last4)


@pytest.mark.parametrize("kind", ref.KINDS)
def test_rest_rows(kind):
    """Rows in no sequence are not read; they stay as they were in a given output and are zeros in a new one."""
    kind = ref.KINDS[kind]
    x = data("rest", 40, kind, "exp")
    lo, hi = x["offsets"][0], x["offsets"][-1]
    rest = torch.ones(300, dtype=torch.bool)
    rest[lo:hi] = False
    for t in (x["a"], x["b"], x["dh"]):
        t[rest.cuda()] = float("nan")
    out = torch.full_like(x["b"], 5.0)
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp")
    sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp", out=out)
    assert (out[rest.cuda()] == 5).all() and (h[rest.cuda()] == 0).all() and torch.equal(out[lo:hi], h[lo:hi])
    h[rest.cuda()] = float("nan")
    da, db = torch.full_like(out, 5.0), torch.full_like(out, 5.0)
    got = sla.sla_recur_adjoint(x["a"], h, x["dh"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate="exp")
    sla.sla_recur_adjoint(x["a"], h, x["dh"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate="exp", da=da, db=db)
    for mine, theirs in zip((da, db), got):
        assert (mine[rest.cuda()] == 5).all() and (theirs[rest.cuda()] == 0).all()
        assert torch.equal(mine[lo:hi], theirs[lo:hi]) and torch.isfinite(theirs).all()
    assert torch.isfinite(last).all() and torch.isfinite(got[2]).all()


def test_not_finite_stays_in_its_channel_and_sequence():
    x = data("ragged", 24, torch.float32, "value")
    clean, _ = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"])
    x["b"][300, 5] = float("nan")
    x["b"][10, 7] = float("inf")
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"])
    assert torch.isnan(h[300:640, 5]).all() and not torch.isfinite(h[10, 7])
    keep = torch.ones_like(h, dtype=torch.bool)
    keep[300:640, 5] = False
    keep[10:131, 7] = False
    assert torch.equal(h[keep], clean[keep])
    # backward: rows in front of it, in its sequence
    clean = sla.sla_recur_adjoint(x["a"], x["b"], x["dh"], h0=x["h0"], seq_off=x["off"])[1]
    x["dh"][200, 3] = float("nan")
    db = sla.sla_recur_adjoint(x["a"], x["b"], x["dh"], h0=x["h0"], seq_off=x["off"])[1]
    assert torch.isnan(db[131:201, 3]).all()
    keep = torch.ones_like(db, dtype=torch.bool)
    keep[131:201, 3] = False
    assert torch.equal(db[keep], clean[keep])


@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("low", [0.3, 0.45])
def test_not_finite_states_stay_over_vanishing_products(kind, value, low):
    """Products of coefficients that leave the range, of either sign, over a few hundred rows: a state that is not
    finite stays so to the end of its sequence, and does not reach the next one."""
    kind = ref.KINDS[kind]
    g = torch.Generator().manual_seed(5)
    tokens, d, border = 2500, 96, 2100
    a = low + (0.9 - low) * torch.rand(tokens, d, generator=g)
    a[torch.rand(tokens, d, generator=g) < 0.5] *= -1
    a = a.to(kind).cuda()
    x = torch.randn(tokens, d, generator=g).to(kind).cuda()
    off = torch.tensor([0, border, tokens], dtype=torch.int32).cuda()
    h0 = torch.zeros(2, d, dtype=ref.wide(kind), device="cuda")
    b = x.clone()
    b[10] = value
    h, last = sla.sla_recur_solve(a, b, h0, off)
    assert h[:10].isfinite().all() and not h[10:border].isfinite().any() and h[border:].isfinite().all()
    assert not last[0].isfinite().any() and last[1].isfinite().all()
    dh = x.clone()
    dh[border - 10] = value
    _, db, dh0 = sla.sla_recur_adjoint(a, x, dh, h0=h0, seq_off=off)
    assert not db[:border - 9].isfinite().any() and db[border - 9:].isfinite().all()
    assert not dh0[0].isfinite().any() and dh0[1].isfinite().all()


def test_partial_gradients():
    x = data("ragged", 56, torch.bfloat16, "sigmoid")
    h, _ = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="sigmoid")
    kw = dict(h0=x["h0"], seq_off=x["off"], gate="sigmoid")
    full = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], dh_last=x["dlast"], **kw)
    no_da = sla.sla_recur_adjoint(x["a"], h, x["dh"], dh_last=x["dlast"], want_da=False, **kw)
    assert no_da[0] is None and torch.equal(no_da[1], full[1]) and torch.equal(no_da[2], full[2])
    no_db = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], dh_last=x["dlast"], want_db=False, **kw)
    assert no_db[1] is None and torch.equal(no_db[0], full[0]) and torch.equal(no_db[2], full[2])
    check_adjoint(x, h, sla.sla_recur_adjoint(x["a"], h, None, b=x["b"], dh_last=x["dlast"], **kw), "sigmoid",
                  torch.bfloat16, dh=False)
    check_adjoint(x, h, sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], **kw), "sigmoid", torch.bfloat16, dlast=False)
    with pytest.raises(ValueError, match="needs b"):
        sla.sla_recur_adjoint(x["a"], h, x["dh"], **kw)
    with pytest.raises(ValueError, match="both"):
        sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], da=torch.empty_like(h), **kw)


@pytest.mark.parametrize("gate", sla.GATES)
@pytest.mark.parametrize("first", [True, False])
def test_gradients_against_differences(gate, first):
    x = data((23, [0, 4, 4, 5, 21]), 3, torch.float64, gate, first=first)
    inputs = [x["a"].requires_grad_(), x["b"].requires_grad_()] + ([x["h0"].requires_grad_()] if first else [])

    def f(a, b, h0=None):
        return sla.recurrence(a, b, h0, x["off"], gate=gate)
    assert torch.autograd.gradcheck(f, inputs, eps=1e-6, atol=1e-7, rtol=1e-6)


def test_autograd_layouts():
    """Broadcast coefficients, a last-state loss alone, transposed inputs, an expanded gradient."""
    B, T, d = 2, 70, 12
    g = torch.Generator().manual_seed(3)
    decay = torch.rand(d, generator=g, dtype=torch.float64).cuda().requires_grad_()
    b = torch.randn(T, B, d, generator=g, dtype=torch.float64).cuda().requires_grad_()
    rows = b.transpose(0, 1)
    h, last = sla.recurrence(decay.expand(B, T, d), rows)
    gd, gb = torch.autograd.grad(h.sum(), [decay, b], retain_graph=True)
    gd2, gb2 = torch.autograd.grad(last.square().sum(), [decay, b])

    def plain():
        v, hs = torch.zeros(B, d, dtype=torch.float64, device="cuda"), []
        for t in range(T):
            v = decay * v + b[t]
            hs.append(v)
        return torch.stack(hs, 1), v
    p, plast = plain()
    wd, wb = torch.autograd.grad(p.sum(), [decay, b], retain_graph=True)
    wd2, wb2 = torch.autograd.grad(plast.square().sum(), [decay, b])
    for got, want in ((gd, wd), (gb, wb), (gd2, wd2), (gb2, wb2)):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-11)
    with pytest.raises(RuntimeError):     # no second derivative is offered
        h, _ = sla.recurrence(decay.expand(B, T, d), rows)
        (x,) = torch.autograd.grad(h.square().sum(), [decay], create_graph=True)
        torch.autograd.grad(x.sum(), [decay])


@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("gate", sla.GATES)
def test_step(kind, gate):
    kind = ref.KINDS[kind]
    for rows, d, slots in ((1, 1, 1), (5, 33, 9), (70, 136, 90), (3, 1000, 3)):
        x = data((rows, [0, rows]), d, kind, gate)
        g = torch.Generator().manual_seed(rows)
        pool = torch.randn(slots, d, generator=g).to(ref.wide(kind)).cuda()
        index = torch.randperm(slots, generator=g)[:rows].to(torch.int32)
        if rows > 2:
            index[-1], index[1] = -1, slots       # padding of the batch, both ways
        state, out = pool.clone(), torch.full_like(x["b"], 5.0)
        h = sla.sla_recur_step(x["a"], x["b"], state, index.cuda(), gate=gate)
        again = pool.clone()
        sla.sla_recur_step(x["a"], x["b"], again, index.cuda(), gate=gate, out=out)
        assert torch.equal(state, again)
        live = ((index >= 0) & (index < slots)).cuda()
        assert (h[~live] == 0).all() and (out[~live] == 5).all() and torch.equal(h[live], out[live])
        at = index.cuda()[live].long()
        want, wlast, e, elast = ref.solve(ref.host(x["a"][live]), ref.host(x["b"][live]), ref.host(pool[at]),
                                          list(range(int(live.sum()) + 1)), gate, kind)
        ref.within(h[live], want, ref.storage(want, e, kind))
        ref.within(state[at], wlast, ref.storage(wlast, elast, ref.wide(kind)))
        others = torch.ones(slots, dtype=torch.bool, device="cuda")
        others[at] = False
        assert torch.equal(state[others], pool[others])


def test_step_layouts_and_refusals():
    rows, d = 6, 40
    x = data((rows, [0, rows]), d, torch.bfloat16, "exp")
    pool = torch.zeros(rows, 3 * d, device="cuda")
    state = pool[:, d:2 * d]
    h = sla.sla_recur_step(x["a"][:1].expand(rows, d), x["b"], state, gate="exp")
    assert torch.equal(h, x["b"]) and torch.equal(state, x["b"].float())
    assert (pool[:, :d] == 0).all() and (pool[:, 2 * d:] == 0).all()
    with pytest.raises(ValueError, match="slot"):
        sla.sla_recur_step(x["a"], x["b"], state[:3])
    with pytest.raises(ValueError, match="state"):
        sla.sla_recur_step(x["a"], x["b"], state.bfloat16())
    with pytest.raises(ValueError, match="index"):
        sla.sla_recur_step(x["a"], x["b"], state, torch.arange(rows, device="cuda"))


def test_steps_are_the_solve():
    """A prompt by the solve, then tokens one at a time: the states of one longer solve."""
    x = data((60, [0, 60]), 64, torch.float32, "sigmoid", first=False)
    h, last = sla.sla_recur_solve(x["a"], x["b"], gate="sigmoid")
    _, state = sla.sla_recur_solve(x["a"][:50], x["b"][:50], gate="sigmoid")
    for t in range(50, 60):
        y = sla.sla_recur_step(x["a"][t:t + 1], x["b"][t:t + 1], state, gate="sigmoid")
        assert torch.allclose(y, h[t:t + 1], rtol=0, atol=1e-5)
    assert torch.allclose(state, last, rtol=0, atol=1e-5)


def test_same_bits_every_time():
    x = data((20000, [0, 777, 15000, 20000]), 200, torch.bfloat16, "exp")
    first = None
    for _ in range(20):
        h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp")
        got = sla.sla_recur_adjoint(x["a"], h, x["dh"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate="exp")
        now = (h, last) + got
        first = first or now
        assert all(torch.equal(p, q) for p, q in zip(first, now))


@pytest.mark.parametrize("channels", [1024, 1022])
def test_many_sequences_many_times(channels):
    """Thousands of short sequences over several tiles a block, again and again: where borders lie takes longer to find
    than a tile's work, so every hand-over between a block's warps is met in another order."""
    tokens, seqs = 12000, 3000
    g = torch.Generator().manual_seed(1)
    cuts = torch.randint(0, tokens + 1, (seqs - 1,), generator=g).sort().values
    off = torch.cat([torch.tensor([0]), cuts, torch.tensor([tokens])]).tolist()
    x = data((tokens, off), channels, torch.bfloat16, "exp")
    few = [0, 5, 1023]
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp")
    few = [c for c in few if c < channels]
    sub = {k: (v[:, few].contiguous() if torch.is_tensor(v) and v.dim() == 2 else v) for k, v in x.items()}
    check_solve(sub, h[:, few], last[:, few], "exp", torch.bfloat16)
    got = sla.sla_recur_adjoint(x["a"], h, x["dh"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate="exp")
    for _ in range(40):
        again = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp")
        assert torch.equal(again[0], h) and torch.equal(again[1], last)
        back = sla.sla_recur_adjoint(x["a"], h, x["dh"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"], gate="exp")
        assert all(torch.equal(s, t) for s, t in zip(back, got))


def test_streams_and_graphs():
    """On a stream given or current, captured, replayed on new inputs, two captured calls at the same time."""
    x = data((9000, [0, 4000, 9000]), 72, torch.bfloat16, "exp")
    y = data((9000, [0, 10, 9000]), 72, torch.bfloat16, "exp", seed=5)

    def both(v):
        h, last = sla.sla_recur_solve(v["a"], v["b"], v["h0"], v["off"], gate="exp")
        return (h, last) + sla.sla_recur_adjoint(v["a"], h, v["dh"], h0=v["h0"], seq_off=v["off"], dh_last=v["dlast"],
                                                 gate="exp")
    want_x, want_y = both(x), both(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h, _ = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp", stream=side)
    h2, _ = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp", stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(h, want_x[0]) and torch.equal(h2, want_x[0])
    fixed = [{k: (v.clone() if torch.is_tensor(v) else v) for k, v in x.items()} for _ in range(2)]
    graphs, outs = [], []
    for v in fixed:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(v))
        graphs.append(g)
    for k in range(4):
        for i, v in enumerate(fixed):
            for name in ("a", "b", "h0", "dh", "dlast", "off"):
                v[name].copy_((x, y)[(k + i) % 2][name])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = (want_x, want_y)[(k + i) % 2]
            assert all(torch.equal(p, q) for p, q in zip(outs[i], want))


def test_rows_beyond_32_bit_offsets():
    """Row offsets past 2^31 elements (and 2^32 bytes): a long strided buffer holds inputs and output."""
    tokens, ld, d = 34000, 65536, 16
    buf = torch.zeros(tokens, ld, dtype=torch.bfloat16, device="cuda")
    x = data((tokens, [0, 30000, tokens]), d, torch.bfloat16, "exp")
    buf[:, :d], buf[:, 1000:1000 + d] = x["a"], x["b"]
    h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate="exp")
    h2, last2 = sla.sla_recur_solve(buf[:, :d], buf[:, 1000:1000 + d], x["h0"], x["off"], gate="exp",
                                    out=buf[:, 2000:2000 + d])
    assert torch.equal(h, h2) and torch.equal(last, last2)
    da, db, dh0 = sla.sla_recur_adjoint(x["a"], h, x["dh"], h0=x["h0"], seq_off=x["off"], gate="exp")
    sla.sla_recur_adjoint(buf[:, :d], h2, x["dh"], h0=x["h0"], seq_off=x["off"], gate="exp",
                          da=buf[:, 3000:3000 + d], db=buf[:, 4000:4000 + d])
    assert torch.equal(buf[:, 3000:3000 + d], da) and torch.equal(buf[:, 4000:4000 + d], db)


def test_nothing_to_do():
    """No tokens, no channels, no sequences; first states pass through to the last ones."""
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    h0 = torch.rand(3, 8, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert torch.equal(sla.sla_recur_solve(z(0, 8), z(0, 8), h0, off)[1], h0)
    assert torch.equal(sla.sla_recur_solve(z(3, 0, 8), z(3, 0, 8), h0)[1], h0)
    assert [t.shape for t in sla.sla_recur_solve(z(0, 5, 8), z(0, 5, 8))] == [(0, 5, 8), (0, 8)]
    assert [t.shape for t in sla.sla_recur_solve(z(5, 0), z(5, 0))] == [(5, 0), (1, 0)]
    da, db, dh0 = sla.sla_recur_adjoint(z(0, 8), z(0, 8), None, h0=h0, seq_off=off, dh_last=2 * h0)
    assert da.shape == db.shape == (0, 8) and torch.equal(dh0, 2 * h0)
    assert sla.sla_recur_step(z(0, 8), z(0, 8), z(0, 8)).shape == (0, 8)
    h = sla.sla_recur_step(z(2, 8) + 1, z(2, 8) + 1, z(0, 8), torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert (h == 0).all()


def test_offsets_out_of_range_stay_inside():
    """Offsets beyond the rows lead to no access outside them (results of such a call are unspecified)."""
    x = data("ragged", 16, torch.float32, "value")
    n = x["off"].numel()
    for bad in ([-5, 2 ** 31 - 1] + [3] * (n - 2), [10 ** 9] * n, list(range(2000, 2000 - n, -1)), [-1] * n):
        off = torch.tensor(bad, dtype=torch.int32).cuda()
        guard = torch.full((720, 16), 5.0, device="cuda")
        sla.sla_recur_solve(x["a"], x["b"], x["h0"], off, out=guard[10:710])
        assert (guard[:10] == 5).all() and (guard[710:] == 5).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_many_steps_of_a_slow_sigmoid_gate(kind):
    """Ten thousand steps at coefficients about 0.9999, inputs of one sign.  Bound: a step rounds its coefficient (1 - w) and its
    sum, u / 2 each below 1 (the sum relative to itself, u), and the weighted input 9 u; every error counts a times in
    the next step.  All of one sign, that is E_t = a E_{t-1} + 1.5 u G_t, besides the inputs' 9 u G_t."""
    kind, d, u = ref.KINDS[kind], 16, 2.0 ** -24
    g = torch.Generator().manual_seed(4)
    rows = 50
    z = torch.log(1 / (2e-4 * torch.rand(rows, d, generator=g, dtype=torch.float64) + 1e-9) - 1).to(kind)
    b = (torch.rand(rows, d, generator=g) + 0.5).to(kind)
    state = torch.zeros(1, d, device="cuda")
    v, err = np.zeros(d), np.zeros(d)
    gz, gb = z.cuda(), b.cuda()
    c, w = ref.gate_of(ref.host(z), "sigmoid")
    for t in range(10000):
        r = t % rows
        sla.sla_recur_step(gz[r:r + 1], gb[r:r + 1], state, gate="sigmoid")
        v = c[r] * v + w[r] * ref.host(b)[r]
        err = c[r] * err + 1.5 * u * v
    ref.within(state, v[None], ref.storage(v, err + 9 * u * v, torch.float32)[None])
