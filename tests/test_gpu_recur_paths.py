"""The recurrence's copies of rows: tensor copies where rows are aligned to 16 bytes, units of 4 bytes or single
values elsewhere.  The arithmetic is the same, so the results have to be the same bits."""
import pytest
import torch

import differentiable_sparse_linear_b200 as sla
import sequence_reference as ref
from test_gpu_recur import data

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
