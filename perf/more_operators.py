"""Timed cases of the experts' operators: tokens sorted by expert and back
with their weights, and the products over groups of rows with bias,
activation and residual, each with its gradient.

`run` is one pass: with `own` through the framework's calls, without it in
elementary torch operations.  Rows that belong to no expert lie behind the
last expert's and stay as they are (zero here).
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, **more):
    return {"name": name, "op": op, **more}


def listed():
    """tokens: T; top: experts of a token; drop: share of the (token, expert)
    pairs that are not routed; ids: integer type of the experts' numbers."""
    return [
        # A decode batch of eight sequences on its way to 64 experts: latency.
        _case("sort_decode", "sort", tokens=8, top=6, experts=64, width=2048, dtype="bf16", ids="i64", drop=0.0),
        # Odd sizes in f32, a seventh of the pairs dropped.
        _case("sort_ragged", "sort", tokens=1009, top=3, experts=37, width=769, dtype="f32", ids="i32", drop=0.14),
        # A training batch, 16 sequences of 1024, the experts of 2048 x 1408.
        _case("sort_batch", "sort", tokens=16384, top=6, experts=64, width=2048, dtype="bf16", ids="i64", drop=0.0),
        # Back from the experts with weights and residual: a decode batch, and the training batch.
        _case("back_decode", "back", tokens=8, top=6, experts=64, width=2048, dtype="bf16", drop=0.0),
        _case("back_batch", "back", tokens=16384, top=6, experts=64, width=2048, dtype="bf16", drop=0.0),
        # Its gradient, for the outputs of the experts and for the weights.
        _case("back_grad_ragged", "back_grad", tokens=1009, top=3, experts=37, width=769, dtype="f32", drop=0.14),
        _case("back_grad_batch", "back_grad", tokens=16384, top=6, experts=64, width=2048, dtype="bf16", drop=0.0),
        # The up product of 64 experts over a decode batch: the weights are read once, for a row or two each.
        _case("linear_decode", "linear", tokens=8, top=6, experts=64, din=2048, dout=1408, dtype="bf16", act="silu",
              bias=False, residual=False, keep=False, drop=0.0),
        # The same over the training batch, with what the gradient needs kept.
        _case("linear_experts", "linear", tokens=16384, top=6, experts=64, din=2048, dout=1408, dtype="bf16",
              act="silu", bias=False, residual=False, keep=True, drop=0.0),
        # A layer of GPT-2 small (the attention's output, with bias and residual), 16 sequences of 1024.
        _case("linear_layer", "linear", tokens=16384, top=1, experts=1, din=768, dout=768, dtype="bf16", act="none",
              bias=True, residual=True, keep=False, drop=0.0),
        # Gradients: odd sizes in f32 over nine groups, and the training batch's experts.
        _case("linear_grad_ragged", "linear_grad", tokens=1501, top=2, experts=9, din=517, dout=259, dtype="f32",
              act="gelu_tanh", bias=True, drop=0.1),
        _case("linear_grad_experts", "linear_grad", tokens=16384, top=6, experts=64, din=2048, dout=1408,
              dtype="bf16", act="silu", bias=False, drop=0.0),
    ]


def draw(rng):
    def size(low, high):
        return int(math.exp(rng.uniform(math.log(low), math.log(high + 0.99))))

    def width(high):
        n = size(8, high)
        return n if rng.random() < 0.25 else -(-n // 8) * 8   # a quarter of them any number

    op = rng.choice(["sort", "back", "back_grad", "linear", "linear", "linear_grad", "linear_grad"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "drop": rng.choice([0.0, 0.0, 0.1, 0.5])}
    experts = rng.choice([1, size(2, 128), size(2, 128)])
    top = 1 if experts == 1 else rng.randint(1, min(8, experts))
    case.update(tokens=size(1, 16384 * 6 // max(top, 6)), top=top, experts=experts)
    if experts == 1:
        case["drop"] = 0.0
    if op == "sort":
        case["ids"] = rng.choice(["i32", "i64"])
    if op in ("sort", "back", "back_grad"):
        case["width"] = width(4096 // (2 if case["dtype"] == "f32" else 1) // 2)
        return case
    case.update(din=width(2048), dout=width(1408), act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                bias=rng.random() < 0.5)
    if op == "linear":
        case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5)
    if case["dtype"] == "f32":   # the f32 rate is a tenth of the bf16 one
        case["tokens"] = max(1, case["tokens"] // 8)
    return case


def _rows(case):
    """Routed (token, expert) pairs, and the experts that have one, as expected."""
    pairs = case["tokens"] * case["top"] * (1 - case["drop"])
    p = case["top"] * (1 - case["drop"]) / case["experts"]
    return pairs, case["experts"] * (1 - (1 - min(p, 1.0)) ** case["tokens"])


def work(case):
    size = {"f32": 4, "bf16": 2}[case["dtype"]]
    slots, (rows, hit), op = case["tokens"] * case["top"], _rows(case), case["op"]
    if op == "sort":
        ids = slots * {"i32": 4, "i64": 8}[case["ids"]]
        return {"bytes": ids + 8 * slots + 4 * case["experts"] + (case["tokens"] + rows) * case["width"] * size,
                "flops": slots}
    if op == "back":
        return {"bytes": (2 * case["tokens"] + rows) * case["width"] * size + 8 * slots,
                "flops": 2 * rows * case["width"]}
    if op == "back_grad":
        return {"bytes": (case["tokens"] + 2 * rows) * case["width"] * size + 12 * slots,
                "flops": 3 * rows * case["width"]}
    din, dout = case["din"], case["dout"]
    if op == "linear":
        outs = 1 + case["residual"] + case["keep"]
        return {"bytes": size * (rows * (din + outs * dout) + hit * dout * (din + case["bias"])),
                "flops": 2 * rows * din * dout}
    acts = 2 if case["act"] != "none" else 1
    return {"bytes": size * (rows * (2 * din + acts * dout) + (hit + case["experts"]) * din * dout
                             + case["bias"] * case["experts"] * dout),
            "flops": 4 * rows * din * dout}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _route(case, gen):
    """(tokens, top) experts of every token, some more often chosen than
    others, and weights that are a softmax over them."""
    e = case["experts"]
    logits = torch.randn(case["tokens"], e, generator=gen, device="cuda")
    logits += 0.5 * torch.sin(torch.arange(e, device="cuda") * 2.4)
    val, ids = torch.topk(logits, case["top"], dim=1)
    if case["drop"]:
        ids[torch.rand(ids.shape, generator=gen, device="cuda") < case["drop"]] = -1
    return ids, torch.softmax(val, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, tokens, top, experts = DTYPES[case["dtype"]], case["tokens"], case["top"], case["experts"]
    slots = tokens * top

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    ids, weights = _route(case, gen)
    s = {"case": dict(case), "op": case["op"]}
    if case["op"] == "sort":
        s["ids"] = ids.to({"i32": torch.int32, "i64": torch.int64}[case["ids"]])
        s["x"] = normal(tokens, case["width"])
        s["xs"] = torch.zeros(slots, case["width"], dtype=dt, device="cuda")
    # What the sort hands on to the calls behind it.
    offsets, order, place = _sort(ids, experts)
    s.update(offsets=offsets, order=order, place=place)
    s["groups"] = offsets if experts > 1 else None   # a layer's product takes all rows
    if case["op"] in ("back", "back_grad"):
        s["weights"] = weights
        s["ys"] = normal(slots, case["width"])
        if case["op"] == "back":
            s["residual"] = normal(tokens, case["width"])
            s["y"] = torch.zeros_like(s["residual"])
        else:
            s["dy"] = normal(tokens, case["width"], std=0.01)
            s["dys"] = torch.zeros_like(s["ys"])
            s["dweights"] = torch.zeros_like(weights)
    if case["op"] in ("linear", "linear_grad"):
        din, dout = case["din"], case["dout"]
        s["counts"] = offsets.tolist()
        s["x"] = normal(slots, din)
        s["w"] = normal(experts, dout, din, std=din ** -0.5)
        s["bias"] = normal(experts, dout, std=0.1) if case["bias"] else None
    if case["op"] == "linear":
        s["residual"] = normal(slots, dout) if case["residual"] else None
        s["y"] = torch.zeros(slots, dout, dtype=dt, device="cuda")
        s["pre"] = torch.zeros_like(s["y"]) if case["keep"] else None
    if case["op"] == "linear_grad":
        s["dy"] = normal(slots, dout, std=0.01)
        s["pre"] = normal(slots, dout) if case["act"] != "none" else None
        s["dx"] = torch.zeros_like(s["x"])
        s["dw"] = torch.zeros_like(s["w"])
        s["db"] = torch.zeros_like(s["bias"]) if case["bias"] else None
    if own and case["op"] in ("back", "back_grad"):
        import dimuon_newton_schulz_amd as D
        s["routes"] = D.ExpertRoutes(offsets, order, place)
    return s


def _sort(ids, experts):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    by_expert, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(experts + 1, device=flat.device)).int()
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=flat.device)
    return (offsets, torch.where(by_expert < experts, order, -1).int(),
            torch.where(key < experts, place, -1).int().view(ids.shape))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0 * z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)


def run(state):
    s, op = state, state["op"]
    case = s["case"]
    if own:
        import dimuon_newton_schulz_amd as D
        if op == "sort":
            routes = D.expert_sort(s["ids"], case["experts"])
            D.expert_gather(s["x"], routes, out=s["xs"])
            return {"offsets": routes.offsets, "order": routes.order, "place": routes.place, "xs": s["xs"]}
        if op == "back":
            return D.expert_combine(s["ys"], s["routes"], weights=s["weights"], residual=s["residual"], out=s["y"])
        if op == "back_grad":
            dys, dweights = D.expert_combine_grad(s["dy"], s["ys"], s["weights"], s["routes"], dys=s["dys"],
                                                  dweights=s["dweights"])
            return {"dys": dys, "dweights": dweights}
        if op == "linear":
            y = D.linear(s["x"], s["w"], bias=s["bias"], activation=case["act"], residual=s["residual"],
                         offsets=s["groups"], pre=s["pre"], out=s["y"])
            return {"y": y, "pre": s["pre"]} if case["keep"] else y
        D.linear_grad(s["dy"], s["x"], s["w"], activation=case["act"], pre=s["pre"], offsets=s["groups"],
                      dx=s["dx"], dw=s["dw"], db=s["db"])
        return _grads(s)
    if op == "sort":
        offsets, order, place = _sort(s["ids"], case["experts"])
        used = place.reshape(-1) >= 0
        token = torch.arange(used.numel(), device=used.device) // case["top"]
        s["xs"][place.reshape(-1)[used].long()] = s["x"][token[used]]
        return {"offsets": offsets, "order": order, "place": place, "xs": s["xs"]}
    if op in ("back", "back_grad"):
        used = s["place"] >= 0
        at = s["place"].clamp(min=0).long()
        if op == "back":
            y = s["residual"].float()
            for j in range(case["top"]):
                rows = s["ys"][at[:, j]].float() * s["weights"][:, j, None]
                y = y + torch.where(used[:, j, None], rows, 0.0)
            s["y"].copy_(y)
            return s["y"]
        dy = s["dy"].float()
        for j in range(case["top"]):
            u = used[:, j]
            s["dys"][at[u, j]] = (dy[u] * s["weights"][u, j, None]).to(s["dys"].dtype)
            s["dweights"][:, j] = torch.where(u, (dy * s["ys"][at[:, j]].float()).sum(1), 0.0)
        return {"dys": s["dys"], "dweights": s["dweights"]}
    for e, (lo, hi) in enumerate(zip(s["counts"][:-1], s["counts"][1:])):
        if op == "linear":
            if lo == hi:
                continue
            z = s["x"][lo:hi].float() @ s["w"][e].float().t()
            if s["bias"] is not None:
                z = z + s["bias"][e].float()
            y = _act(case["act"], z)
            if s["residual"] is not None:
                y = y + s["residual"][lo:hi].float()
            s["y"][lo:hi] = y.to(s["y"].dtype)
            if case["keep"]:
                s["pre"][lo:hi] = z.to(s["y"].dtype)
            continue
        dz = s["dy"][lo:hi].float()
        if s["pre"] is not None:
            dz = dz * _act_slope(case["act"], s["pre"][lo:hi].float())
        s["dx"][lo:hi] = (dz @ s["w"][e].float()).to(s["dx"].dtype)
        s["dw"][e] = (dz.t() @ s["x"][lo:hi].float()).to(s["dw"].dtype)
        if s["db"] is not None:
            s["db"][e] = dz.sum(0).to(s["db"].dtype)
    if op == "linear":
        return {"y": s["y"], "pre": s["pre"]} if case["keep"] else s["y"]
    return _grads(s)


def _grads(s):
    out = {"dx": s["dx"], "dw": s["dw"]}
    if s["db"] is not None:
        out["db"] = s["db"]
    return out


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _phi(z, order):
    """Distribution function of the standard normal (order 0), its density (order 1)."""
    return torch.special.ndtr(z) if order == 0 else torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def _exact_act(name, z, slope):
    if name == "none":
        return torch.ones_like(z) if slope else z
    if name == "relu":
        return torch.heaviside(z, torch.zeros_like(z)) if slope else z.clamp(min=0)
    if name == "gelu":
        return _phi(z, 0) + z * _phi(z, 1) if slope else z * _phi(z, 0)
    # z times a sigmoid of u(z): u = z (silu), or 2 sqrt(2/pi) (z + 0.044715 z^3), since (1 + tanh(u/2)) / 2 = sigmoid(u)
    c = 0.0 if name == "silu" else 0.044715
    k = 1.0 if name == "silu" else math.sqrt(8 / math.pi)
    sig = torch.sigmoid(k * (z + c * z.pow(3)))
    if not slope:
        return z * sig
    return sig + z * sig * (1 - sig) * k * (1 + 3 * c * z.pow(2))


def exact(case, seed):
    s = prepare(case, seed)
    tokens, top, experts, op = case["tokens"], case["top"], case["experts"], case["op"]
    if op == "sort":
        ids = s["ids"].reshape(-1).long().cpu()
        lists = [torch.nonzero(ids == e).view(-1) for e in range(experts)]
        order = torch.cat(lists)
        offsets = torch.tensor([0] + [len(x) for x in lists]).cumsum(0)
        place = torch.full((tokens * top,), -1)
        place[order] = torch.arange(len(order))
        xs = torch.zeros(tokens * top, case["width"], dtype=torch.float64, device="cuda")
        xs[:len(order)] = s["x"].double().index_select(0, torch.div(order, top, rounding_mode="floor").cuda())
        order = torch.cat([order, torch.full((tokens * top - len(order),), -1)])
        return {"offsets": offsets.int().cuda(), "order": order.int().cuda(),
                "place": place.view(tokens, top).int().cuda(), "xs": xs}
    if op in ("back", "back_grad"):
        n = int(s["offsets"][-1])
        slot = s["order"][:n].long()
        token, w = slot // top, s["weights"].reshape(-1)[slot].double()[:, None]
        ys = s["ys"][:n].double()
        if op == "back":
            return s["residual"].double().index_add_(0, token, ys * w)
        dy = s["dy"].double()[token]
        dys = torch.zeros(s["ys"].shape, dtype=torch.float64, device="cuda")
        dys[:n] = dy * w
        dweights = torch.zeros(tokens * top, dtype=torch.float64, device="cuda")
        dweights[slot] = (dy * ys).sum(1)
        return {"dys": dys, "dweights": dweights.view(tokens, top)}
    bounds = s["offsets"].tolist()
    x, w = s["x"].double(), s["w"].double()
    out = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda")
           for k in ("y", "pre", "dx", "dw", "db") if s.get(k) is not None and not (op == "linear_grad" and k == "pre")}
    for e in range(experts):
        r = slice(bounds[e], bounds[e + 1])
        if op == "linear":
            z = torch.mm(x[r], w[e].T)
            if s["bias"] is not None:
                z += s["bias"][e].double()
            out["y"][r] = _exact_act(case["act"], z, False)
            if s["residual"] is not None:
                out["y"][r] += s["residual"][r].double()
            if "pre" in out:
                out["pre"][r] = z
            continue
        dz = s["dy"][r].double()
        if s["pre"] is not None:
            dz = dz * _exact_act(case["act"], s["pre"][r].double(), True)
        out["dx"][r] = torch.mm(dz, w[e])
        out["dw"][e] = torch.mm(dz.T, x[r])
        if "db" in out:
            out["db"][e] = torch.mv(dz.T, torch.ones(len(dz), dtype=torch.float64, device="cuda"))
    if op == "linear":
        return out if case["keep"] else out["y"]
    return out
