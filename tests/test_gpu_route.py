"""Routing of tokens to experts on the GPU: the plan against a sort on the host (equal), the products
and their adjoints against 64-bit sums.

Bounds: a weighted row is one product (u relative) and its rounding; a sum of k terms of magnitude
sum m has error (2k + 1) u m at most, one of n products in any order 2 n u m, u = 2^-24 (2^-53)."""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_b200 as sla
import sequence_reference as ref

pytestmark = pytest.mark.gpu


def choices(tokens, top_k, experts, seed=0, skew=1.0, dropped=0.0, repeat=False):
    g = np.random.default_rng(seed)
    p = np.exp(skew * g.standard_normal(experts))
    p /= p.sum()
    ids = g.choice(experts, size=(tokens, top_k), p=p) if repeat or top_k > experts else np.stack(
        [g.permutation(experts)[:top_k] for _ in range(tokens)]) if tokens else np.zeros((0, top_k), np.int64)
    ids = ids.astype(np.int64)
    if dropped:
        ids[g.random(ids.shape) < dropped] = -1
        ids[g.random(ids.shape) < dropped / 2] = experts
        ids[g.random(ids.shape) < dropped / 2] = 2 ** 31 - 1
    return ids


SORTS = [
    # tokens, top_k, experts, align, dropped
    (0, 2, 4, 1, 0), (1, 1, 1, 1, 0), (1, 1, 5, 1, 1.0), (1, 8, 64, 16, 0), (7, 3, 5, 4, 0.2), (16, 4, 64, 1, 0),
    (31, 1, 2, 1, 0), (33, 2, 300, 128, 0.1), (1000, 2, 8, 128, 0.05), (1024, 1, 1, 1, 0), (4097, 3, 17, 1, 0.3),
    (5000, 8, 256, 64, 0), (20011, 5, 100, 1, 0.01), (300, 2, 4096, 2, 0), (9000, 4, 4096, 1, 0.1), (65536, 8, 128, 128, 0),
    (200000, 2, 33, 1, 0), (70000, 1, 1000, 8, 0.5), (1500, 2, 4096, 2, 0.1), (250000, 5, 40, 1, 0.02),
]


@pytest.mark.parametrize("tokens,top_k,experts,align,dropped", SORTS)
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_sort(tokens, top_k, experts, align, dropped, kind):
    ids = choices(tokens, top_k, experts, seed=tokens + experts, dropped=dropped, repeat=tokens > 3000)
    slots = tokens * top_k + experts * (align - 1)
    for extra in (0, 13):
        r = sla.sla_route_sort(torch.from_numpy(ids).to(kind).cuda(), experts, align=align,
                               n_slots=slots + extra if extra else None)
        want = ref.sort(ids, experts, align, slots + extra)
        for got, w, name in zip((r.offsets, r.counts, r.entry, r.slot), want, ("offsets", "counts", "entry", "slot")):
            assert np.array_equal(got.cpu().numpy(), w), name


def test_sort_ids_beyond_32_bits_are_dropped():
    ids = torch.tensor([[0, 2 ** 32], [2 ** 32 + 1, 1], [-(2 ** 32), 2]], device="cuda")
    r = sla.sla_route_sort(ids, 3)
    assert r.slot.tolist() == [[0, -1], [-1, 1], [-1, 2]] and r.counts.tolist() == [1, 1, 1]


def test_sort_one_popular_expert():
    ids = np.full((40000, 2), 3, np.int64)
    ids[::1000] = 0
    r = sla.sla_route_sort(torch.from_numpy(ids).cuda(), 5, align=8)
    want = ref.sort(ids, 5, 8, ids.size + 35)
    assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip((r.offsets, r.counts, r.entry, r.slot), want))


def test_sort_of_a_vector_and_refusals():
    ids = torch.tensor([2, 0, 2, 1], device="cuda")
    r = sla.sla_route_sort(ids, 3)
    assert r.slot.tolist() == [[2], [0], [3], [1]] and r.entry.tolist() == [1, 3, 0, 2]
    for bad in (lambda: sla.sla_route_sort(ids.float(), 3), lambda: sla.sla_route_sort(ids[::2], 3),
                lambda: sla.sla_route_sort(ids, 0), lambda: sla.sla_route_sort(ids, 3, align=0),
                lambda: sla.sla_route_sort(ids[None, None], 3)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sla.SlaError):
        sla.sla_route_sort(ids, 3, n_slots=3)
    with pytest.raises(sla.SlaError):
        sla.sla_route_sort(ids, 5000)


PRODUCTS = [
    # tokens, top_k, experts, channels, align, dropped
    (1, 1, 1, 1, 1, 0), (1, 2, 4, 8, 16, 0), (5, 3, 4, 33, 1, 0.3), (64, 2, 8, 64, 8, 0.1), (40, 8, 16, 130, 1, 0),
    (9, 1, 3, 1000, 4, 0), (300, 4, 7, 24, 128, 0.5), (3, 2, 2, 4097, 1, 0), (17, 11, 40, 100, 2, 0.2), (6, 2, 4, 16, 1, 1.0),
    (130, 2, 5, 514, 3, 0.1), (2, 40, 50, 12, 1, 0.1),
]


def problem(tokens, top_k, experts, channels, align, dropped, kind, seed=0):
    ids = choices(tokens, top_k, experts, seed=seed + tokens, dropped=dropped)
    r = sla.sla_route_sort(torch.from_numpy(ids).cuda(), experts, align=align)
    g = torch.Generator().manual_seed(seed)
    return dict(route=r, slot=r.slot.cpu().numpy(), slots=r.n_slots, used=int(r.offsets[-1]),
                x=torch.randn(tokens, channels, generator=g).to(kind).cuda(),
                xs=torch.randn(r.n_slots, channels, generator=g).to(kind).cuda(),
                weight=torch.randn(tokens, top_k, generator=g).to(ref.wide(kind)).cuda())


def check_to_slots(got, p, w, kind, used=None):
    want = ref.to_slots(ref.host(p["x"]), p["slot"], None if w is None else ref.host(w), p["slots"])
    u = 0 if w is None else ref.unit(kind)
    bound = u * np.abs(want) if w is None else ref.storage(want, u * np.abs(want), kind)
    n = p["slots"] if used is None else used
    ref.within(got[:n], want[:n], bound[:n])


def check_to_tokens(got, p, w, kind, top_k):
    want, mag = ref.to_tokens(ref.host(p["xs"]), p["slot"], None if w is None else ref.host(w))
    ref.within(got, want, ref.storage(want, (2 * top_k + 1) * ref.unit(kind) * mag, kind))


def check_pattern(got, p, kind):
    want, mag = ref.on_pattern(ref.host(p["x"]), ref.host(p["xs"]), p["slot"])
    n = p["x"].shape[1]
    e = 2 * n * ref.unit(kind) * mag
    ref.within(got, want, ref.storage(want, e, ref.wide(kind)))


@pytest.mark.parametrize("tokens,top_k,experts,channels,align,dropped", PRODUCTS)
@pytest.mark.parametrize("kind", ref.KINDS)
def test_products(tokens, top_k, experts, channels, align, dropped, kind):
    kind = ref.KINDS[kind]
    p = problem(tokens, top_k, experts, channels, align, dropped, kind)
    r, xs = p["route"], p["xs"].clone()
    # rows of slots without an entry are not read
    free = torch.from_numpy(np.setdiff1d(np.arange(p["slots"]), p["slot"][p["slot"] >= 0])).cuda()
    p["xs"][free] = float("nan")
    for w in (None, p["weight"]):
        check_to_slots(sla.sla_route_dispatch(p["x"], r, w), p, w, kind)
        check_to_tokens(sla.sla_route_combine(p["xs"], r, w), p, w, kind, top_k)
        dx, none = sla.sla_route_dispatch_adjoint(p["xs"], r, weight=w)
        assert none is None
        check_to_tokens(dx, p, w, kind, top_k)
        dx, dw = sla.sla_route_dispatch_adjoint(p["xs"], r, p["x"], w)
        check_to_tokens(dx, p, w, kind, top_k)
        check_pattern(dw, p, kind)
        dys, none = sla.sla_route_combine_adjoint(p["x"], r, weight=w)
        assert none is None
        check_to_slots(dys, p, w, kind)
        dys, dw = sla.sla_route_combine_adjoint(p["x"], r, p["xs"], w)
        check_to_slots(dys, p, w, kind)
        check_pattern(dw, p, kind)
        # a given output: slots behind the experts' stay as they were
        out = torch.full_like(xs, 5.0)
        sla.sla_route_dispatch(p["x"], r, w, out=out)
        check_to_slots(out, p, w, kind, used=p["used"])
        assert (out[p["used"]:] == 5).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_strided_rows(kind):
    kind = ref.KINDS[kind]
    for channels, pad in ((64, 64), (40, 3), (33, 1)):
        p = problem(50, 3, 6, channels, 4, 0.1, kind)
        r, w = p["route"], p["weight"]
        wide = lambda t: torch.cat([t, torch.zeros(t.shape[0], pad, dtype=kind, device="cuda")], 1)[:, :channels]  # noqa: E731
        want = sla.sla_route_dispatch(p["x"], r, w)
        buf = torch.full((p["slots"], channels + pad), 5.0, dtype=kind, device="cuda")
        got = sla.sla_route_dispatch(wide(p["x"]), r, w, out=buf[:, pad:])
        used = p["used"]
        assert torch.equal(got[:used], want[:used]) and (buf[:, :pad] == 5).all()
        assert torch.equal(sla.sla_route_combine(wide(p["xs"]), r, w), sla.sla_route_combine(p["xs"], r, w))
        one = p["x"][:1].expand(50, channels)
        assert torch.equal(sla.sla_route_dispatch(one, r, w), sla.sla_route_dispatch(one.contiguous(), r, w))
        for f, q in ((sla.sla_route_dispatch_adjoint, ("xs", "x")), (sla.sla_route_combine_adjoint, ("x", "xs"))):
            (rows, dw), (rows2, dw2) = f(wide(p[q[0]]), r, wide(p[q[1]]), w), f(p[q[0]], r, p[q[1]], w)
            assert torch.equal(rows, rows2)
            # the dot products run over the channels in an order that goes by the rows' alignment: two sums of
            # the same n products differ by rounding, each within the 2 n u m of any order
            check_pattern(dw, p, kind)
            check_pattern(dw2, p, kind)


def test_nothing_to_do():
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    r = sla.sla_route_sort(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), 3)
    assert sla.sla_route_dispatch(z(4, 0), r).shape == (8, 0) and sla.sla_route_combine(z(8, 0), r).shape == (4, 0)
    assert (sla.sla_route_combine_adjoint(z(4, 0), r, z(8, 0))[1] == 0).all()
    assert (sla.sla_route_dispatch_adjoint(z(8, 0), r, z(4, 0))[1] == 0).all()
    r = sla.sla_route_sort(torch.zeros(0, 2, dtype=torch.int64, device="cuda"), 3, align=4)
    assert r.offsets.tolist() == [0, 0, 0, 0] and (r.entry == -1).all()
    assert (sla.sla_route_dispatch(z(0, 8), r) == 0).all() and sla.sla_route_combine(z(9, 8), r).shape == (0, 8)


def test_slots_out_of_range_stay_inside():
    """A plan whose slots lead outside the rows reads and writes nothing there."""
    p = problem(20, 2, 4, 32, 1, 0, torch.float32)
    r = p["route"]
    slot = r.slot.clone()
    slot[3, 0], slot[4, 1], slot[5, 0] = 40, 2 ** 31 - 1, -7
    bad = sla.Route(r.offsets, r.counts, r.entry, slot)
    guard = torch.full((60, 32), 5.0, device="cuda")
    sla.sla_route_dispatch(p["x"], bad, out=guard[10:50])
    assert (guard[:10] == 5).all() and (guard[50:] == 5).all()
    y = sla.sla_route_combine(p["xs"], bad)
    assert torch.equal(y[3], p["xs"][slot[3, 1].item()]) and torch.equal(y[4], p["xs"][slot[4, 0].item()])
    for counts, offsets in ((r.counts * 100, r.offsets * 100), (r.counts * 0 - 9, r.offsets * 0 - 5)):
        guard.fill_(5.0)
        sla.sla_route_dispatch(p["x"], sla.Route(offsets, counts, r.entry, r.slot), out=guard[10:50])
        assert (guard[:10] == 5).all() and (guard[50:] == 5).all()


def test_gradients_against_differences():
    ids = torch.from_numpy(choices(6, 2, 4, dropped=0.2)).cuda()
    r = sla.sla_route_sort(ids, 4, align=2)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(6, 5, generator=g, dtype=torch.float64).cuda().requires_grad_()
    xs = torch.randn(r.n_slots, 5, generator=g, dtype=torch.float64).cuda().requires_grad_()
    w = torch.randn(6, 2, generator=g, dtype=torch.float64).cuda().requires_grad_()
    for f, inputs in ((lambda x: sla.route_dispatch(x, r), (x,)), (lambda x, w: sla.route_dispatch(x, r, w), (x, w)),
                      (lambda y: sla.route_combine(y, r), (xs,)), (lambda y, w: sla.route_combine(y, r, w), (xs, w))):
        assert torch.autograd.gradcheck(f, inputs, eps=1e-6, atol=1e-7, rtol=1e-6)


def test_same_bits_streams_and_graphs():
    p = problem(3000, 4, 32, 264, 16, 0.05, torch.bfloat16)
    ids = torch.from_numpy(choices(3000, 4, 32, seed=3000, dropped=0.05)).cuda()

    def both():
        r = sla.sla_route_sort(ids, 32, align=16)
        return (r.offsets, r.counts, r.entry, r.slot, sla.sla_route_dispatch(p["x"], r, p["weight"]),
                sla.sla_route_combine(p["xs"], r, p["weight"]),
                *sla.sla_route_combine_adjoint(p["x"], r, p["xs"], p["weight"]),
                *sla.sla_route_dispatch_adjoint(p["xs"], r, p["x"], p["weight"]))
    want = both()
    for _ in range(5):
        assert all(torch.equal(s, t) for s, t in zip(both(), want))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = sla.sla_route_combine(p["xs"], p["route"], p["weight"], stream=side)
    r = sla.sla_route_sort(ids, 32, align=16, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want[5]) and torch.equal(r.slot, want[3])
    g = torch.cuda.CUDAGraph()
    kept = ids.clone()
    with torch.cuda.graph(g):
        got = both()
    ids.copy_(kept.flip(0))
    g.replay()
    flipped = both()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(got, flipped))
    ids.copy_(kept)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(got, want))


def test_rows_beyond_32_bit_offsets():
    """Slot rows past 2^31 elements and 2^32 bytes."""
    tokens, ld, channels = 17000, 65536, 24
    ids = torch.from_numpy(choices(tokens, 2, 8, repeat=True)).cuda()
    r = sla.sla_route_sort(ids, 8)
    x = torch.randn(tokens, channels, device="cuda").bfloat16()
    w = torch.rand(tokens, 2, device="cuda")
    buf = torch.zeros(2 * tokens, ld, dtype=torch.bfloat16, device="cuda")
    view = buf[:, 64:64 + channels]
    sla.sla_route_dispatch(x, r, w, out=view)
    want = sla.sla_route_dispatch(x, r, w)
    assert torch.equal(view, want)
    assert torch.equal(sla.sla_route_combine(view, r, w), sla.sla_route_combine(want, r, w))


def test_sorts_from_several_host_threads():
    """Calls of different expert counts at the same time through the C ABI, which releases the interpreter's lock: a call
    changes nothing that another one's launch needs."""
    import threading

    from differentiable_sparse_linear_b200 import _lib
    lib = _lib.load()
    wrong, start = [], threading.Barrier(4)

    def work(experts, top_k, seed):
        stream = torch.cuda.Stream()
        ids = choices(6000, top_k, experts, seed=seed, repeat=True)
        n = ids.size
        want = ref.sort(ids, experts, 1, n)
        with torch.cuda.stream(stream):
            d = torch.from_numpy(ids).cuda()
            out = [torch.empty(s, dtype=torch.int32, device="cuda") for s in (experts + 1, experts, n, n)]
            size = lib.sla_route_workspace_bytes(6000, top_k, experts)
            mem = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
            stream.synchronize()
            start.wait()
            for _ in range(4000):
                s = lib.sla_route_sort(6000, top_k, experts, 1, d.data_ptr(), 8, n, *[t.data_ptr() for t in out], mem.data_ptr(),
                                       size, stream.cuda_stream)
                if s:
                    wrong.append((experts, s, lib.sla_last_error()))
                    return
            stream.synchronize()
            if not all(np.array_equal(t.cpu().numpy(), w.reshape(-1)) for t, w in zip(out, want)):
                wrong.append((experts, "result"))
    threads = [threading.Thread(target=work, args=a) for a in ((4096, 2, 1), (1000, 2, 2), (4096, 1, 3), (700, 1, 4))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
