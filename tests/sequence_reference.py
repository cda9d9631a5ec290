"""Plain 64-bit forms of the sequence operators on the host, one row after the other, and the error
bounds that the GPU tests hold the kernels to.

Error bounds.  With u the unit roundoff of the arithmetic (2^-24 for fp32, 2^-53 for fp64) a row of
the recurrence h_t = a_t h_{t-1} + w_t b_t takes: the coefficient from its gate (exp: the function's
2 ulp = 4u; sigmoid: that, an addition, a quotient and a product: 8u), the weighted input (8u and
one product: 9u), and the sum (u, or 2u more where a partial result of a split axis is rounded in
between, twice).  All of it is relative to G_t = |a_t| G_{t-1} + |w_t b_t|, which bounds every
partial sum, so the error obeys E_t = |a_t| E_{t-1} + 24 u G_t to first order.  A row is rounded to its
storage type once: half a step, eps/2 relative, or half the smallest subnormal.
"""
import numpy as np
import torch

KINDS = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}


def unit(kind):
    return 2.0 ** -53 if kind == torch.float64 else 2.0 ** -24


def wide(kind):
    return torch.float64 if kind == torch.float64 else torch.float32


def host(t):
    return t.detach().double().cpu().numpy()


def storage(x, err, kind):
    """Bound on the distance of a stored value from x, with err before the rounding."""
    tiny = 2.0 ** -25 if kind == torch.float16 else torch.finfo(kind).tiny * torch.finfo(kind).eps
    return err + torch.finfo(kind).eps / 2 * (np.abs(x) + err) + tiny


def gate_of(z, gate):
    if gate == "value":
        return z, np.ones_like(z)
    if gate == "exp":
        return np.exp(z), np.ones_like(z)
    e = np.exp(-np.abs(z))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(z < 0, small, big), np.where(z < 0, big, small)


def solve(a, b, h0, off, gate, kind):
    """(h, last, bound of h before rounding, bound of last) of packed rows; rows in no sequence are 0."""
    tokens, d = b.shape
    k = 24 * unit(kind)
    h, e = np.zeros((tokens, d)), np.zeros((tokens, d))
    last, elast = np.zeros((len(off) - 1, d)), np.zeros((len(off) - 1, d))
    for s in range(len(off) - 1):
        v = np.zeros(d) if h0 is None else h0[s].copy()
        g, err = np.abs(v), np.zeros(d)
        for t in range(off[s], off[s + 1]):
            c, w = gate_of(a[t], gate)
            if t == off[s] and h0 is None:
                c = np.zeros(d)
            v = c * v + w * b[t]
            g = np.abs(c) * g + np.abs(w * b[t])
            err = np.abs(c) * err + k * g
            h[t], e[t] = v, err
        last[s], elast[s] = v, err
    return h, last, e, elast


def adjoint(a, b, h, h0, dh, dlast, off, gate, kind):
    """{name: (value, bound before rounding)} of da, db, dh0; h: the rows as stored."""
    tokens, d = a.shape
    u = unit(kind)
    k = 24 * u
    da, db, eda, edb = (np.zeros((tokens, d)) for _ in range(4))
    dh0, edh0 = np.zeros((len(off) - 1, d)), np.zeros((len(off) - 1, d))
    for s in range(len(off) - 1):
        carry = np.zeros(d) if dlast is None else dlast[s].copy()
        g, err = np.abs(carry), np.zeros(d)
        for t in range(off[s + 1] - 1, off[s] - 1, -1):
            c, w = gate_of(a[t], gate)
            x = np.zeros(d) if dh is None else dh[t]
            lam = x + carry
            g = np.abs(x) + g
            err = err + k * g
            before = h[t - 1] if t > off[s] else (np.zeros(d) if h0 is None else h0[s])
            db[t], edb[t] = w * lam, w * err + 24 * u * w * g
            if gate == "value":
                f, m = before, np.abs(before)
            elif gate == "exp":
                f, m = before * c, np.abs(before) * c
            else:
                f, m = (before - b[t]) * c * w, (np.abs(before) + np.abs(b[t])) * c * w
            da[t], eda[t] = lam * f, m * err + 24 * u * m * g
            carry, g, err = c * lam, np.abs(c) * g, np.abs(c) * err + k * np.abs(c) * g
        dh0[s], edh0[s] = carry, err
    return dict(da=(da, eda), db=(db, edb), dh0=(dh0, edh0))


def sort(ids, experts, align, slots):
    """(offsets, counts, entry, slot) of [tokens, top_k] ids."""
    flat = ids.reshape(-1)
    offsets, counts = [0], []
    entry, slot = np.full(slots, -1, np.int32), np.full(flat.shape, -1, np.int32)
    for x in range(experts):
        mine = np.nonzero(flat == x)[0]
        at = offsets[-1]
        entry[at:at + len(mine)] = mine
        slot[mine] = at + np.arange(len(mine))
        counts.append(len(mine))
        offsets.append(at + -(-len(mine) // align) * align)
    return (np.array(offsets, np.int32), np.array(counts, np.int32), entry, slot.reshape(ids.shape))


def to_slots(x, slot, weight, slots):
    """R^T x in 64 bits; rows of slots without an entry are 0."""
    out = np.zeros((slots, x.shape[1]))
    for t, j in zip(*np.nonzero(slot >= 0)):
        out[slot[t, j]] = x[t] * (1 if weight is None else weight[t, j])
    return out


def to_tokens(xs, slot, weight):
    """(R xs, sum of the terms' magnitudes)."""
    out, mag = np.zeros((slot.shape[0], xs.shape[1])), np.zeros((slot.shape[0], xs.shape[1]))
    for t, j in zip(*np.nonzero(slot >= 0)):
        term = xs[slot[t, j]] * (1 if weight is None else weight[t, j])
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def on_pattern(x, xs, slot):
    """(x . xs on the pattern, sum of the terms' magnitudes)."""
    out, mag = np.zeros(slot.shape), np.zeros(slot.shape)
    for t, j in zip(*np.nonzero(slot >= 0)):
        out[t, j] = x[t] @ xs[slot[t, j]]
        mag[t, j] = np.abs(x[t]) @ np.abs(xs[slot[t, j]])
    return out, mag


def within(got, want, bound):
    """Every element of the tensor within its bound (and equal where not finite)."""
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (got.shape, want.shape)
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} values off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]}, bound {np.broadcast_to(bound, want.shape)[bad][0]}")
