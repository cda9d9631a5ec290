"""The sequence operators run together, as a block of a model uses them: a gated recurrence over packed
sequences, its rows sent to experts, the experts' products, the weighted sum back and a residual;
trained (gradients of every parameter), served token by token, and captured."""
import pytest
import torch

import differentiable_sparse_linear_b200 as sla

pytestmark = pytest.mark.gpu

D, E, K = 16, 4, 2


def parameters(dtype):
    g = torch.Generator().manual_seed(11)
    shapes = dict(gate=(D, D), inp=(D, D), router=(D, E), experts=(E, D, D))
    return {k: (torch.randn(s, generator=g, dtype=torch.float64) / D ** 0.5).to(dtype).cuda().requires_grad_()
            for k, s in shapes.items()}


def experts_of(xs, route, w, dtype):
    """Every expert's product on its own slots, as a dense product masked by the plan."""
    rows = torch.arange(xs.shape[0], device=xs.device)
    mine = (rows[None] >= route.offsets[:-1, None]) & (rows[None] < route.offsets[1:, None])
    return torch.einsum("es,sd,edf->sf", mine.to(dtype), xs, w)


def block(x, p, off, h0):
    h, last = sla.recurrence(x @ p["gate"], x @ p["inp"], h0, off, gate="sigmoid")
    prob, ids = torch.softmax(h @ p["router"], -1).topk(K, dim=-1)
    route = sla.sla_route_sort(ids, E, align=4)
    xs = sla.route_dispatch(h, route)
    y = sla.route_combine(torch.tanh(experts_of(xs, route, p["experts"], x.dtype)), route,
                          prob.to(torch.float64 if x.dtype == torch.float64 else torch.float32))
    return x + y, last, ids


def plain(x, p, offsets, h0):
    z, u = x @ p["gate"], x @ p["inp"]
    c = torch.sigmoid(z)
    hs, lasts = [], []
    for s in range(len(offsets) - 1):
        v = h0[s]
        for t in range(offsets[s], offsets[s + 1]):
            v = c[t] * v + (1 - c[t]) * u[t]
            hs.append(v)
        lasts.append(v)
    h = torch.stack(hs)
    prob, ids = torch.softmax(h @ p["router"], -1).topk(K, dim=-1)
    y = sum(prob[:, j, None] * torch.tanh(torch.einsum("td,tdf->tf", h, p["experts"][ids[:, j]])) for j in range(K))
    return x + y, torch.stack(lasts), ids


def test_block_and_its_gradients():
    offsets = [0, 9, 9, 40, 77]
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(2)
    x = torch.randn(77, D, generator=g, dtype=torch.float64).cuda().requires_grad_()
    h0 = torch.randn(4, D, generator=g, dtype=torch.float64).cuda().requires_grad_()
    p = parameters(torch.float64)
    wanted = [x, h0, *p.values()]
    y, last, ids = block(x, p, off, h0)
    z, zlast, zids = plain(x, p, offsets, h0)
    assert torch.equal(ids, zids)
    assert torch.allclose(y, z, rtol=1e-11, atol=1e-12) and torch.allclose(last, zlast, rtol=1e-11, atol=1e-12)
    c = torch.randn(77, D, generator=g, dtype=torch.float64).cuda()
    got = torch.autograd.grad((y * c).sum() + last.square().sum(), wanted)
    want = torch.autograd.grad((z * c).sum() + zlast.square().sum(), wanted)
    for s, t in zip(got, want):
        assert torch.allclose(s, t, rtol=1e-9, atol=1e-10)


def test_block_trains_in_16_bits():
    off = torch.tensor([0, 100, 256], dtype=torch.int32).cuda()
    p = parameters(torch.bfloat16)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(256, D, generator=g).bfloat16().cuda()
    opt = torch.optim.SGD(list(p.values()), lr=0.01)
    for _ in range(3):
        opt.zero_grad()
        y, _, _ = block(x, p, off, None)
        y.float().square().mean().backward()
        assert all(t.grad is not None and torch.isfinite(t.grad).all() for t in p.values())
        opt.step()


def test_prompt_then_tokens():
    """A prompt by the solve, then one token at a time through the step and the same routing, against one long pass."""
    p = {k: t.detach() for k, t in parameters(torch.float64).items()}
    g = torch.Generator().manual_seed(6)
    x = torch.randn(2, 40, D, generator=g, dtype=torch.float64).cuda()
    off = torch.tensor([0, 40, 80], dtype=torch.int32).cuda()
    with torch.no_grad():
        want, _, _ = block(x.reshape(80, D), p, off, None)
        want = want.view(2, 40, D)
        _, pool = sla.sla_recur_solve(x[:, :30].contiguous() @ p["gate"], x[:, :30].contiguous() @ p["inp"], gate="sigmoid")
        for t in range(30, 40):
            h = sla.sla_recur_step(x[:, t] @ p["gate"], x[:, t] @ p["inp"], pool, gate="sigmoid")
            prob, ids = torch.softmax(h @ p["router"], -1).topk(K, dim=-1)
            route = sla.sla_route_sort(ids, E)
            y = sla.sla_route_combine(torch.tanh(experts_of(sla.sla_route_dispatch(h, route), route, p["experts"],
                                                            torch.float64)), route, prob)
            assert torch.allclose(x[:, t] + y, want[:, t], rtol=1e-10, atol=1e-11)


def test_block_captured():
    """The whole block forward and backward in one graph, replayed on new rows and new lengths."""
    p = {k: t.detach() for k, t in parameters(torch.float32).items()}
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(300, D, generator=g).cuda() for _ in range(2)]
    offs = [torch.tensor(o, dtype=torch.int32).cuda() for o in ([0, 100, 300], [0, 299, 300])]

    def step(x, off):
        q = {k: t.detach().requires_grad_() for k, t in p.items()}
        y, last, _ = block(x, q, off, None)
        return (y, last) + torch.autograd.grad(y.square().mean(), list(q.values()))
    want = [step(x, o) for x, o in zip(xs, offs)]
    x, off = xs[0].clone(), offs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, off)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, off)
    for k in (1, 0, 1):
        x.copy_(xs[k])
        off.copy_(offs[k])
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(got, want[k]):
            assert torch.allclose(s, t, rtol=1e-4, atol=1e-6)
