"""The recurrence's copies of rows: tensor copies where rows are aligned to 16 bytes, units of 4 bytes or single
values elsewhere.  The arithmetic is the same, so the results have to be the same bits."""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_b200 as sla
import sequence_reference as ref
from test_gpu_recur import check_adjoint, check_solve, data

pytestmark = pytest.mark.gpu


def pitched(t, ld):
    """The same rows, ld elements apart."""
    buf = torch.zeros(t.shape[0], ld, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("gate", sla.GATES)
@pytest.mark.parametrize("d", [1000, 517])
def test_rows_without_alignment_give_the_aligned_bits(kind, gate, d):
    """Rows of units of 4 bytes (an even pitch of 16-bit values) and of single values (an odd one), many tiles a
    block, again and again: outputs go through the shared memory that the next tiles' copies overwrite."""
    kind = ref.KINDS[kind]
    x = data((6000, [0, 2500, 2501, 5900]), d, kind, gate)

    def both(ld):
        v = {k: pitched(t, ld) if torch.is_tensor(t) and t.dim() == 2 and t.shape[0] == 6000 else t for k, t in x.items()}
        like = lambda: pitched(torch.zeros_like(x["b"]), ld)  # noqa: E731
        h, last = sla.sla_recur_solve(v["a"], v["b"], v["h0"], v["off"], gate=gate, out=like())
        out = sla.sla_recur_adjoint(v["a"], h, v["dh"], b=v["b"], h0=v["h0"], seq_off=v["off"], dh_last=v["dlast"],
                                    gate=gate, da=like(), db=like())
        return (h, last) + out
    want = both(d + 16 - d % 16)
    for ld in (d + 18 - d % 2, d + 17 - d % 2):
        for _ in range(5):
            got = both(ld)
            assert all(torch.equal(p, q) for p, q in zip(got, want))


# rows of a tile: forward, backward, backward with the sigmoid gate
TILES = (176, 160, 144)


@pytest.mark.parametrize("rows", TILES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("gate", sla.GATES)
def test_ends_and_borders_at_tile_ends(rows, kind, gate):
    """Totals of a tile, two and three, one row more or less, and borders there, counted from either end (backward
    tiles are counted from the last row)."""
    kind = ref.KINDS[kind]
    for tokens, off in ([(n * rows + k, [0, n * rows + k]) for n in (1, 2) for k in (-1, 0, 1)] +
                        [(3 * rows + k, [0, rows + m, 2 * rows + m, 3 * rows + k]) for k in (0, 5) for m in (-1, 0, 1)] +
                        [(3 * rows + 5, [0, rows + m + 5, 2 * rows + m + 5, 3 * rows + 5]) for m in (-1, 0, 1)] +
                        [(3 * rows, [rows, rows, 2 * rows, 2 * rows]), (3 * rows, [rows - 1, rows, 2 * rows, 2 * rows + 1])]):
        for d in (40, 33):
            x = data((tokens, off), d, kind, gate)
            h, last = sla.sla_recur_solve(x["a"], x["b"], x["h0"], x["off"], gate=gate)
            check_solve(x, h, last, gate, kind)
            got = sla.sla_recur_adjoint(x["a"], h, x["dh"], b=x["b"], h0=x["h0"], seq_off=x["off"], dh_last=x["dlast"],
                                        gate=gate)
            check_adjoint(x, h, got, gate, kind)


@pytest.mark.parametrize("gate,kind", [("value", "f32"), ("value", "f64"), ("sigmoid", "f32"), ("exp", "bf16")])
@pytest.mark.parametrize("back", [False, True])
def test_long_memory(gate, kind, back):
    """Coefficients about 0.9999, inputs of one sign: a state is what ten thousand rows left.

    Bound.  u = 2^-24 (2^-53).  A row takes part in at most six roundings on the way to its state: the product inside
    its run of four rows and the sum there (two backward), the products and sums of runs and tiles (fewer than one
    each a row).  Each is at most u relative to the partial state G_t (all terms are positive).  Taken as
    independent and zero in the mean, their effect at a row has the variance V_t <= a^2 V_{t-1} + 6 (u G_t)^2 / 3 (a
    rounding is spread over [-u, u]), and the chance of a deviation of 8 standard deviations is below 2 exp(-32), 1e-8
    for all values together.  Added with one sign, u / 2 each below 1: the three products of a run, whose last
    digits (1 - a)(1 - a') are below half a step and always dropped; a coefficient from a gate, rounded once (1 - w,
    or 1 plus a series that drops z^2 / 2).  And the weighted input's 9 u.  Against 24 u a row that is 30 to 60 times
    tighter."""
    kind = ref.KINDS[kind]
    T, d, u = 40000, 12, ref.unit(kind)
    g = torch.Generator().manual_seed(11)
    far = 2e-4 * torch.rand(T, d, generator=g, dtype=torch.float64) + 1e-9    # 1 - a
    a = {"value": 1 - far, "exp": torch.log1p(-far), "sigmoid": torch.log((1 - far) / far)}[gate].to(kind)
    b = (torch.rand(T, d, generator=g) + 0.5).to(kind)
    if back:                                               # lambda_t = b_t + a_{t+1} lambda_{t+1}; db = w lambda
        z = torch.zeros(T, d, dtype=kind, device="cuda")
        _, got, end = sla.sla_recur_adjoint(a.cuda(), z, b.cuda(), b=z, h0=torch.zeros(1, d, dtype=ref.wide(kind), device="cuda"),
                                            gate=gate)
    else:
        got, end = sla.sla_recur_solve(a.cuda(), b.cuda(), gate=gate)
    c, w = ref.gate_of(ref.host(a), gate)
    x = ref.host(b)
    want, bound, v, var, lin = np.zeros((T, d)), np.zeros((T, d)), np.zeros(d), np.zeros(d), np.zeros(d)
    k = u * (3 / 8 if gate == "value" else 7 / 8)
    for t in (range(T - 1, -1, -1) if back else range(T)):
        if back:                                           # v is e = a lambda of the row behind
            lam = x[t] + v
            want[t], bound[t] = w[t] * lam, w[t] * (8 * np.sqrt(var) + lin + 9 * u * lam)
            v = c[t] * lam
            var, lin = c[t] ** 2 * (var + 2 * (u * lam) ** 2), c[t] * (lin + k * lam)
        else:
            v = c[t] * v + w[t] * x[t]
            var, lin = c[t] ** 2 * var + 2 * (u * v) ** 2, c[t] * lin + k * v
            want[t], bound[t] = v, 8 * np.sqrt(var) + lin + 9 * u * v
    ref.within(got, want, ref.storage(want, bound, kind))
    ref.within(end, v[None], ref.storage(v, 8 * np.sqrt(var) + lin + 9 * u * v, ref.wide(kind))[None])
