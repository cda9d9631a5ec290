"""Measured cases of the sequence operators: the gated linear recurrence (its solve, its adjoint
and its single-token step) and the routing of tokens to experts (the sort, the products with the
routing matrix and its transpose, and their gradients on the pattern).

`run` computes a case in plain torch operations (32-bit arithmetic, one rounding at the end)
where `own` is false and by the library's operators where it is true; `exact` computes it
from the definition in 64 bits.

Layouts.  A packed batch of sequences is [tokens, channels] with int32 offsets; rows behind the
last sequence belong to no sequence and come back as zeros.  Recurrent states are 32-bit.  A routing
plan is what the sort returns: per-expert offsets and counts, `entry` (slot -> token * top_k + choice,
-1 where a slot only pads an expert's rows) and `slot` (the inverse, -1 where a choice was dropped).
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZES = {"f32": 4, "f64": 8, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of a small model: a handful of sequences, latency is all there is
        dict(name="step_4x512_f32", op="step", rows=4, channels=512, slots=8, type="f32", gate="value"),
        # a serving batch: rows of a state pool picked by index, some rows of the batch are padding
        dict(name="step_384x4096_bf16", op="step", rows=384, channels=4096, slots=512, type="bf16", gate="sigmoid"),
        # a short prompt, fp32
        dict(name="solve_200x384_f32", op="solve", tokens=200, channels=384, seqs=1, type="f32", gate="value", tail=0),
        # a training batch of packed documents, long ones and short ones
        dict(name="solve_65536x4096_bf16", op="solve", tokens=65536, channels=4096, seqs=24, type="bf16", gate="exp", tail=100),
        # backward pass on odd sizes
        dict(name="adjoint_3001x1001_f32", op="adjoint", tokens=3001, channels=1001, seqs=7, type="f32", gate="sigmoid", tail=9),
        # backward pass of one long document
        dict(name="adjoint_32768x2560_bf16", op="adjoint", tokens=32768, channels=2560, seqs=1, type="bf16", gate="exp", tail=0),
        # routing of a decoding batch
        dict(name="sort_16x4_e64", op="sort", tokens=16, top_k=4, experts=64, align=1, drop=0),
        # routing of a training batch, experts' rows padded to the tile of a product
        dict(name="sort_131072x8_e256", op="sort", tokens=131072, top_k=8, experts=256, align=128, drop=1000),
        # tokens of a decoding batch to their experts
        dict(name="dispatch_8x2_1024_bf16", op="dispatch", tokens=8, top_k=2, experts=8, channels=1024, align=1, type="bf16", weighted=False, drop=0),
        # tokens of a training batch to their experts, experts' rows padded
        dict(name="dispatch_16384x2_4096_bf16", op="dispatch", tokens=16384, top_k=2, experts=64, channels=4096, align=128, type="bf16", weighted=False, drop=64),
        # experts' answers back, odd sizes
        dict(name="combine_3001x3_1025_f32", op="combine", tokens=3001, top_k=3, experts=17, channels=1025, align=1, type="f32", weighted=True, drop=10),
        # backward pass of the weighted sum: gradients of the experts' answers and of the weights
        dict(name="combine_grad_16384x4_2048_bf16", op="combine_grad", tokens=16384, top_k=4, experts=128, channels=2048, align=1, type="bf16", weighted=True, drop=0),
    ]


def _span(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("step", "solve", "solve", "adjoint", "adjoint", "sort", "dispatch", "combine", "dispatch_grad", "combine_grad"))
    kind = rng.choice(("bf16", "bf16", "f16", "f32"))
    gate = rng.choice(("value", "exp", "sigmoid"))
    channels = _span(rng, 48, 6000)
    if rng.random() < 0.7:  # model widths are multiples of a power of two more often than not
        channels = max(64, channels // 64 * 64)
    if op == "step":
        rows = _span(rng, 1, 768)
        return dict(op=op, rows=rows, channels=channels, slots=rows + rng.randint(0, rows), type=kind, gate=gate)
    if op in ("solve", "adjoint"):
        tokens = _span(rng, 1, min(100000, (1 << 27) // channels))
        return dict(op=op, tokens=tokens, channels=channels, seqs=_span(rng, 1, max(1, tokens // 2)) if rng.random() < 0.6 else 1,
                    type=kind, gate=gate, tail=rng.choice((0, 0, rng.randint(0, tokens // 8))))
    top_k = rng.randint(1, 8)
    experts = _span(rng, top_k, 256)
    align = rng.choice((1, 1, 16, 128))
    if op == "sort":
        tokens = _span(rng, 1, 100000)
        return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, align=align, drop=rng.choice((0, rng.randint(0, tokens // 8))))
    tokens = _span(rng, 1, max(1, min(50000, (1 << 27) // (channels * top_k))))
    return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, channels=channels, align=align, type=kind,
                weighted=op.startswith("combine") or rng.random() < 0.3, drop=rng.choice((0, rng.randint(0, tokens // 8))))


def work(case):
    op = case["op"]
    if op == "sort":
        n = case["tokens"] * case["top_k"]
        slots = _slots(case)
        # ids read (64-bit), slot written, entry written, offsets and counts written
        return {"bytes": 8 * n + 4 * n + 4 * slots + 8 * case["experts"] + 4, "flops": 0}
    s, d = _SIZES[case["type"]], case["channels"]
    if op == "step":
        # coefficients, inputs and outputs once; the 32-bit states of the rows read and written
        return {"bytes": case["rows"] * d * (3 * s + 8) + 4 * case["rows"], "flops": 2 * case["rows"] * d}
    if op in ("solve", "adjoint"):
        n, state = (case["tokens"] - case["tail"]) * d, 4 * case["seqs"] * d
        if op == "solve":
            # a, b read; h written; first and last states
            return {"bytes": 2 * n * s + case["tokens"] * d * s + 2 * state, "flops": 2 * n}
        reads = 4 if case["gate"] == "sigmoid" else 3
        # a, h, dh (and b for the sigmoid gate) read; da, db written; h0, dh_last, dh0
        return {"bytes": reads * n * s + 2 * case["tokens"] * d * s + 3 * state, "flops": 4 * n}
    live = case["tokens"] - case["drop"]
    pairs, slots = live * case["top_k"], _slots(case)
    plan = 4 * case["tokens"] * case["top_k"] + (4 * case["tokens"] * case["top_k"] if case["weighted"] else 0)
    row = d * s
    if op == "dispatch":  # every live token's row read once, every slot's row written once
        return {"bytes": live * row + slots * row + plan, "flops": pairs * d if case["weighted"] else 0}
    if op == "combine":  # the used slots' rows read once, every token's row written once
        return {"bytes": pairs * row + case["tokens"] * row + plan, "flops": 2 * pairs * d}
    weights = 4 * case["tokens"] * case["top_k"] if case["weighted"] else 0
    if op == "dispatch_grad":  # dxs (and x) read, dx (and dweight) written
        return {"bytes": pairs * row + case["tokens"] * row + (live * row if case["weighted"] else 0) + plan + weights,
                "flops": (4 if case["weighted"] else 1) * pairs * d}
    # combine_grad: dy and ys read, dys and dweight written
    return {"bytes": live * row + pairs * row + slots * row + plan + weights, "flops": 3 * pairs * d}


# ------------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Lengths of the packed sequences: uneven, some of them empty where there are many."""
    r = random.Random(seed * 7 + 1)
    total, seqs = case["tokens"] - case["tail"], case["seqs"]
    cuts = sorted(r.randint(0, total) for _ in range(seqs - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _gate_input(shape, gate, kind, g):
    """What a gate layer gives: coefficients near 1 with a spread of time scales over the channels."""
    scale = torch.rand(shape[-1], generator=g, device="cuda") * 5 + 0.5
    z = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(0.8).add_(scale)
    if gate == "sigmoid":
        return z.to(kind)
    decay = torch.nn.functional.softplus(-z)                 # -log sigmoid(z)
    return (decay.neg_() if gate == "exp" else decay.neg_().exp_()).to(kind)


def _slots(case):
    return case["tokens"] * case["top_k"] + case["experts"] * (case["align"] - 1)


def _experts(case, g):
    """The router's choices (64-bit, as a top-k gives them): popular experts and rare ones; the last
    `drop` tokens are padding of the batch and go nowhere."""
    tokens, experts = case["tokens"], case["experts"]
    bias = torch.randn(experts, generator=g, device="cuda")
    logits = torch.randn((tokens, experts), generator=g, device="cuda") + bias
    ids = logits.topk(case["top_k"], dim=1).indices
    if case["drop"]:
        ids[tokens - case["drop"]:] = -1
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    if op == "sort":
        return dict(case=case, expert=_experts(case, g))
    kind = _TYPES[case["type"]]
    if op == "step":
        rows, d, slots = case["rows"], case["channels"], case["slots"]
        index = torch.randperm(slots, generator=g, device="cuda")[:rows].to(torch.int32)
        if rows >= 16:
            index[rows - rows // 16:] = -1                   # padding rows of the batch
        return dict(case=case, a=_gate_input((rows, d), case["gate"], kind, g), b=normal(rows, d).to(kind),
                    state=normal(slots, d), index=index)
    if op in ("solve", "adjoint"):
        tokens, d = case["tokens"], case["channels"]
        lengths = _lengths(case, int(seed))
        ends = torch.tensor(lengths).cumsum(0)
        off = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).cuda()
        s = dict(case=case, off=off, longest=max(lengths), a=_gate_input((tokens, d), case["gate"], kind, g),
                 b=normal(tokens, d).to(kind), h0=normal(case["seqs"], d))
        if op == "adjoint":
            s["h"] = _plain_solve(s["a"], s["b"], s["h0"], off, s["longest"], case["gate"])[0]
            s["dh"], s["dlast"] = normal(tokens, d).to(kind), normal(case["seqs"], d)
        return s
    tokens, d, k = case["tokens"], case["channels"], case["top_k"]
    plan = _plain_sort(_experts(case, g), case["experts"], case["align"], _slots(case))
    s = dict(case=case, plan=plan, weight=torch.rand((tokens, k), generator=g, device="cuda") if case["weighted"] else None)
    if op in ("dispatch", "dispatch_grad", "combine_grad"):
        s["x"] = normal(tokens, d).to(kind)                  # token side: x, or dy
    if op in ("combine", "dispatch_grad", "combine_grad"):
        s["xs"] = normal(_slots(case), d).to(kind)           # slot side: ys, or dxs
    return s


# ------------------------------------------------------------------------------------ the pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import differentiable_sparse_linear_b200 as sla
    case = s["case"]
    op = case["op"]
    if op == "step":
        h = sla.sla_recur_step(s["a"], s["b"], s["state"], s["index"], gate=case["gate"])
        return dict(h=h, state=s["state"])
    if op == "solve":
        h, last = sla.sla_recur_solve(s["a"], s["b"], s["h0"], s["off"], gate=case["gate"])
        return dict(h=h, last=last)
    if op == "adjoint":
        da, db, dh0 = sla.sla_recur_adjoint(s["a"], s["h"], s["dh"], b=s["b"] if case["gate"] == "sigmoid" else None,
                                            h0=s["h0"], seq_off=s["off"], dh_last=s["dlast"], gate=case["gate"])
        return dict(da=da, db=db, dh0=dh0)
    if op == "sort":
        r = sla.sla_route_sort(s["expert"], case["experts"], align=case["align"])
        return dict(offsets=r.offsets, counts=r.counts, entry=r.entry, slot=r.slot)
    p = s["plan"]
    route = sla.Route(offsets=p["offsets"], counts=p["counts"], entry=p["entry"], slot=p["slot"])
    if op == "dispatch":
        return dict(xs=sla.sla_route_dispatch(s["x"], route, s["weight"]))
    if op == "combine":
        return dict(y=sla.sla_route_combine(s["xs"], route, s["weight"]))
    if op == "dispatch_grad":
        dx, dw = sla.sla_route_dispatch_adjoint(s["xs"], route, s["x"] if case["weighted"] else None, s["weight"])
        return dict(dx=dx, dweight=dw) if case["weighted"] else dict(dx=dx)
    dys, dw = sla.sla_route_combine_adjoint(s["x"], route, s["xs"], s["weight"])
    return dict(dys=dys, dweight=dw)


# ------------------------------------------------------------------------------------ plain forms

def _coefficients(a, b, gate):
    """(a_t, u_t) of h_t = a_t h_{t-1} + u_t in 32 bits."""
    a, b = a.float(), b.float()
    if gate == "value":
        return a, b
    if gate == "exp":
        return torch.exp(a), b
    return torch.sigmoid(a), torch.sigmoid(-a) * b


def _bounds(off, tokens):
    """Masks [tokens, 1] of rows that start a sequence and of rows inside one, and each row's sequence."""
    rows = torch.arange(tokens, device=off.device)
    seq = torch.searchsorted(off[1:].contiguous(), rows.to(off.dtype), right=True)
    inside = (rows >= off[0]) & (rows < off[-1])
    seq = seq.clamp(max=off.numel() - 2)
    start = inside & (rows == off[seq])
    return start[:, None], inside[:, None], seq


def _scan(a, u, longest):
    """h_t = a_t h_{t-1} + u_t along the first axis by doubling; a is zero where a sequence starts."""
    d = 1
    while d < longest:
        u[d:] = u[d:] + a[d:] * u[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return u


def _plain_solve(a, b, h0, off, longest, gate):
    kind, tokens = b.dtype, b.shape[0]
    start, inside, seq = _bounds(off, tokens)
    c, u = _coefficients(a, b, gate)
    u = torch.where(start, u + c * h0[seq], u)
    u = torch.where(inside, u, 0.0)
    c = torch.where(start | ~inside, 0.0, c)
    h = _scan(c, u, longest)
    full = off[1:] > off[:-1]
    last = torch.where(full[:, None], h[(off[1:] - 1).clamp(min=0).long()], h0)
    return h.to(kind), last


def _plain_adjoint(a, b, h0, h, dh, dlast, off, longest, gate):
    kind, tokens = h.dtype, h.shape[0]
    start, inside, seq = _bounds(off, tokens)
    c, _ = _coefficients(a, b, gate)
    rows = torch.arange(tokens, device=a.device)[:, None]
    end = inside & (rows + 1 == off[1:][seq][:, None])
    nxt = torch.cat([c[1:], torch.zeros_like(c[:1])])        # the coefficient that carries row t into row t + 1
    nxt = torch.where(end | ~inside, 0.0, nxt)
    grad = torch.where(inside, dh.float(), 0.0)
    grad = torch.where(end, grad + dlast[seq], grad)
    lam = _scan(nxt.flip(0), grad.flip(0), longest).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]]).float()
    before = torch.where(start, h0[seq], before)
    before = torch.where(inside, before, 0.0)
    if gate == "value":
        da, db = lam * before, lam
    elif gate == "exp":
        da, db = lam * before * c, lam
    else:
        rest = torch.sigmoid(-a.float())
        da = torch.where(inside, lam * (before - b.float()) * c * rest, 0.0)
        db = lam * rest
    full = off[1:] > off[:-1]
    first = off[:-1].long().clamp(max=tokens - 1)
    dh0 = torch.where(full[:, None], lam[first] * c[first], dlast)
    return da.to(kind), db.to(kind), dh0


def _plain_step(a, b, state, index, gate):
    c, u = _coefficients(a, b, gate)
    live = ((index >= 0) & (index < state.shape[0]))[:, None]
    at = index.clamp(min=0).long()
    h = c * state[at] + u
    # rows of padding write nothing: they go to a row that is cut off again
    out = torch.cat([state, state[:1]])
    out[torch.where(live[:, 0], at, state.shape[0])] = h
    state.copy_(out[:-1])
    return torch.where(live, h, 0.0).to(b.dtype)


def _plain_sort(expert, experts, align, slots):
    flat = expert.reshape(-1)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    before = counts.cumsum(0) - counts
    rows = (counts[:experts] + align - 1) // align * align
    offsets = torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0)])
    key = key[order]
    place = offsets[key] + torch.arange(n, device=flat.device) - before[key]
    live = key < experts
    entry = torch.full((slots + 1,), -1, dtype=torch.int64, device=flat.device)
    entry[torch.where(live, place, slots)] = torch.where(live, order, -1)
    slot = torch.empty_like(flat)
    slot[order] = torch.where(live, place, -1)
    small = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(offsets=small(offsets), counts=small(counts[:experts]), entry=small(entry[:slots]), slot=small(slot.reshape(expert.shape)))


def _to_slots(x, plan, weight):
    """R^T x: every slot gets its token's row, times its weight; slots of padding get zeros."""
    entry, k = plan["entry"].long(), plan["slot"].shape[1]
    live = (entry >= 0)[:, None]
    at = entry.clamp(min=0)
    rows = x.float()[at // k]
    if weight is not None:
        rows = rows * weight.reshape(-1)[at][:, None]
    return torch.where(live, rows, 0.0)


def _to_tokens(xs, plan, weight):
    """R xs: every token's sum over its slots, times their weights."""
    slot = plan["slot"].long()
    live = (slot >= 0)[:, :, None]
    rows = torch.where(live, xs[slot.clamp(min=0)].float(), 0.0)
    if weight is not None:
        rows = rows * weight[:, :, None]
    return rows.sum(1)


def _on_pattern(x, xs, plan):
    """x . xs for every (token, choice) that has a slot, 0 for the others."""
    slot = plan["slot"].long()
    dots = (xs[slot.clamp(min=0)].float() * x.float()[:, None, :]).sum(2)
    return torch.where(slot >= 0, dots, 0.0)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "step":
        return dict(h=_plain_step(s["a"], s["b"], s["state"], s["index"], case["gate"]), state=s["state"])
    if op == "solve":
        h, last = _plain_solve(s["a"], s["b"], s["h0"], s["off"], s["longest"], case["gate"])
        return dict(h=h, last=last)
    if op == "adjoint":
        da, db, dh0 = _plain_adjoint(s["a"], s["b"], s["h0"], s["h"], s["dh"], s["dlast"], s["off"], s["longest"], case["gate"])
        return dict(da=da, db=db, dh0=dh0)
    if op == "sort":
        return _plain_sort(s["expert"], case["experts"], case["align"], _slots(case))
    plan, weight = s["plan"], s["weight"]
    kind = _TYPES[case["type"]]
    if op == "dispatch":
        return dict(xs=_to_slots(s["x"], plan, weight).to(kind))
    if op == "combine":
        return dict(y=_to_tokens(s["xs"], plan, weight).to(kind))
    if op == "dispatch_grad":
        dx = _to_tokens(s["xs"], plan, weight).to(kind)
        return dict(dx=dx, dweight=_on_pattern(s["x"], s["xs"], plan)) if case["weighted"] else dict(dx=dx)
    return dict(dys=_to_slots(s["x"], plan, weight).to(kind), dweight=_on_pattern(s["x"], s["xs"], plan))


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The outputs of `run` from the definitions, one token (or one routed pair) after the other, in 64 bits."""
    op = case["op"]
    if op == "sort":
        return None                                          # whole numbers only
    s = prepare(case, seed)
    if op in ("step", "solve", "adjoint"):
        wide = lambda t: t.to(torch.float64)  # noqa: E731

        def gate_of(rows_a):
            z = wide(rows_a)
            if case["gate"] == "value":
                return z, torch.ones_like(z)
            if case["gate"] == "exp":
                return z.exp(), torch.ones_like(z)
            return 1 / (1 + (-z).exp()), 1 / (1 + z.exp())

        if op == "step":
            state, h = wide(s["state"]), torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
            for r, i in enumerate(s["index"].tolist()):
                if 0 <= i < state.shape[0]:
                    c, w = gate_of(s["a"][r])
                    state[i] = c * state[i] + w * wide(s["b"][r])
                    h[r] = state[i]
            return dict(h=h, state=state)
        off = s["off"].tolist()
        tokens, d = s["b"].shape
        # sequences longest first: step j advances those that have a row j, which are the first ones
        order = sorted(range(len(off) - 1), key=lambda i: off[i] - off[i + 1])
        starts = torch.tensor([off[i] for i in order], device="cuda")
        lengths = [off[i + 1] - off[i] for i in order]
        inverse = torch.tensor(sorted(range(len(order)), key=lambda i: order[i]), device="cuda")
        pick = torch.tensor(order, device="cuda")
        live = len(order)
        if op == "solve":
            h = torch.zeros((tokens, d), dtype=torch.float64, device="cuda")
            now = wide(s["h0"])[pick]
            for j in range(lengths[0]):
                while lengths[live - 1] <= j:
                    live -= 1
                rows = starts[:live] + j
                c, w = gate_of(s["a"][rows])
                now[:live] = c * now[:live] + w * wide(s["b"][rows])
                h[rows] = now[:live]
            return dict(h=h, last=now[inverse])
        da = torch.zeros((tokens, d), dtype=torch.float64, device="cuda")
        db = torch.zeros_like(da)
        carry = wide(s["dlast"])[pick]                       # d loss / d (state behind the row at hand)
        ends = starts + torch.tensor(lengths, device="cuda")
        h0 = wide(s["h0"])[pick]
        for j in range(lengths[0]):                          # j rows before the end
            while lengths[live - 1] <= j:
                live -= 1
            rows = ends[:live] - 1 - j
            c, w = gate_of(s["a"][rows])
            lam = wide(s["dh"][rows]) + carry[:live]
            first = (rows == starts[:live])[:, None]
            before = torch.where(first, h0[:live], wide(s["h"][(rows - 1).clamp(min=0)]))
            if case["gate"] == "value":
                da[rows] = lam * before
            elif case["gate"] == "exp":
                da[rows] = lam * before * c
            else:
                da[rows] = lam * (before - wide(s["b"][rows])) * c * w
            db[rows] = lam * w
            carry[:live] = lam * c
        return dict(da=da, db=db, dh0=carry[inverse])
    # routing: one choice of every token at a time
    plan, tokens, d = s["plan"], case["tokens"], case["channels"]
    weight = s["weight"].double() if case["weighted"] else torch.ones((tokens, case["top_k"]), dtype=torch.float64, device="cuda")
    out_tokens = torch.zeros((tokens, d), dtype=torch.float64, device="cuda")
    out_slots = torch.zeros((_slots(case), d), dtype=torch.float64, device="cuda")
    dots = torch.zeros((tokens, case["top_k"]), dtype=torch.float64, device="cuda")
    for j in range(case["top_k"]):
        slot = plan["slot"][:, j].long()
        who = torch.nonzero(slot >= 0)[:, 0]
        slot = slot[who]
        if op in ("dispatch", "combine_grad"):
            out_slots[slot] = weight[who, j, None] * s["x"][who].double()
        else:
            out_tokens[who] += weight[who, j, None] * s["xs"][slot].double()
        if op == "combine_grad" or (op == "dispatch_grad" and case["weighted"]):
            dots[who, j] = (s["x"][who].double() * s["xs"][slot].double()).sum(1)
    if op == "dispatch":
        return dict(xs=out_slots)
    if op == "combine":
        return dict(y=out_tokens)
    if op == "dispatch_grad":
        return dict(dx=out_tokens, dweight=dots) if case["weighted"] else dict(dx=out_tokens)
    return dict(dys=out_slots, dweight=dots)
