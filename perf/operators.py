"""Timed cases of the AdamW operators: the step with 32-bit and with 8-bit
moments over many tensors at once, the moments as values (saving and loading
them), and the global gradient norm with its clip coefficient.

A case's tensors live in flat buffers, each tensor starting at a multiple of
256 elements, as a program with flat parameter buffers holds them; the gaps
hold zeros.  `run` is one pass: with `own` through the framework's plans,
without it in elementary torch operations over the flat buffers.
"""

import math

import torch

own = False

BLOCK = 256              # elements that share a scale of the 8-bit moments
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.1
MAX_VECTOR = 8192        # tensors up to this size are vectors (norms, biases): no weight decay
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, sizes, **more):
    return {"name": name, "op": op, "sizes": sizes, **more}


def listed():
    """sizes: element counts, largest first; AxB is A tensors of B elements."""
    embed = "38597376,786432,50x768"            # GPT-2 small: 50257 x 768 embedding, 1024 positions, 25 norms
    experts = "128x2883584"                     # 64 experts of 2048 x 1408, up and down
    lora = "128x32768"                          # 64 pairs of 8 x 4096 and 4096 x 8
    return [
        # The norm weights and biases of GPT-2 small, f32: one short launch.
        _case("adamw_norms", "adamw", "50x768", w="f32", g="f32", master=False, clip=True, step=1),
        # What Muon leaves over in GPT-2 small, mixed precision with f32 master weights.
        _case("adamw_embed_master", "adamw", embed, w="bf16", g="bf16", master=True, clip=True, step=250),
        # Odd sizes, from one element up: a small model in f32.
        _case("adamw_ragged", "adamw", "1000003,517251,40000,4097,1023,257,31,7,1", w="f32", g="f32", master=False,
              clip=False, step=40),
        # A full expert set, bf16 weights and gradients.
        _case("adamw_experts", "adamw", experts, w="bf16", g="bf16", master=False, clip=False, step=1000),
        # LoRA factors under AdamW with 8-bit moments: a short call.
        _case("adamw8_lora", "adamw8", lora, w="bf16", g="bf16", master=False, clip=True, rounding="stochastic",
              step=10),
        # What Muon leaves over in GPT-2 small, 8-bit moments, f32 master weights.
        _case("adamw8_embed", "adamw8", embed, w="bf16", g="bf16", master=True, clip=True, rounding="stochastic",
              step=250),
        # Odd sizes, nearest rounding, f32 weights.
        _case("adamw8_ragged", "adamw8", "1000003,517251,40000,4097,1023,257,31,7,1", w="f32", g="f32", master=False,
              clip=False, rounding="nearest", step=40),
        # A full expert set, 8-bit moments.
        _case("adamw8_experts", "adamw8", experts, w="bf16", g="bf16", master=False, clip=False,
              rounding="stochastic", step=1000),
        # Saving 8-bit moments as f32 values.
        _case("state_save", "save", embed, values="f32"),
        # Loading f32 moments of an expert set into 8 bits, and reading back what they now stand for.
        _case("state_load", "load", experts, values="f32"),
        # The clip norm of a LoRA set (a short call) and of a full expert set.
        _case("norm_lora", "norm", lora, g="f32"),
        _case("norm_experts", "norm", experts, g="bf16"),
    ]


def draw(rng):
    op = rng.choice(["adamw", "adamw", "adamw8", "adamw8", "save", "load", "norm"])
    groups, room = [], 360_000_000   # elements
    for _ in range(rng.randint(1, 4)):
        n = min(room, int(math.exp(rng.uniform(0.0, math.log(2.0e8)))))
        if n < 1:
            break
        groups.append((n, int(math.exp(rng.uniform(0.0, math.log(min(128, room // n) + 0.5))))))
        room -= n * groups[-1][1]
    groups.sort(reverse=True)
    case = {"op": op, "sizes": ",".join("%dx%d" % (c, n) for n, c in groups)}
    if op in ("adamw", "adamw8"):
        w = rng.choice(["f32", "bf16"])
        case.update(w=w, g=rng.choice(["f32", "bf16"]), master=w == "bf16" and rng.random() < 0.4,
                    clip=rng.random() < 0.5, step=int(math.exp(rng.uniform(0.0, math.log(50000.0)))))
    if op == "adamw8":
        case["rounding"] = rng.choice(["stochastic", "stochastic", "nearest"])
    if op in ("save", "load"):
        case["values"] = rng.choice(["f32", "bf16"])
    if op == "norm":
        case["g"] = rng.choice(["f32", "bf16"])
    return case


def _sizes(case):
    out = []
    for part in case["sizes"].split(","):
        count, _, n = part.rpartition("x")
        out += [int(n)] * int(count or 1)
    return out


def _layout(sizes):
    """Offset of every tensor in the flat buffers, and the buffers' length."""
    offsets, at = [], 0
    for n in sizes:
        offsets.append(at)
        at += -(-n // BLOCK) * BLOCK
    return offsets, at


def work(case):
    n = sum(_sizes(case))
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    scales = 8 * n / BLOCK
    if op == "norm":
        return {"bytes": n * size[case["g"]], "flops": 2 * n}
    if op == "save":
        return {"bytes": n * (2 + 2 * size[case["values"]]) + scales, "flops": 2 * n}
    if op == "load":
        return {"bytes": n * (2 * size[case["values"]] + 2 + 4) + scales, "flops": 8 * n}
    w = size[case["w"]]
    per = size[case["g"]] + (w + 8 if case["master"] else 2 * w)
    if op == "adamw":
        return {"bytes": n * (per + 16), "flops": 16 * n}
    return {"bytes": n * (per + 4 + 4) + 2 * scales, "flops": 40 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _values(case, seed):
    """(w, g, m, v) in float32 over the flat buffers, zero in the gaps.
    Magnitudes spread over a few decades; a part of the embedding-like tensors
    has never seen a gradient (its moments are zero too)."""
    sizes = _sizes(case)
    offsets, total = _layout(sizes)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(std):
        return torch.randn(total, generator=gen, device="cuda") * std

    used = (torch.rand(total // BLOCK, generator=gen, device="cuda") > 0.1).float().repeat_interleave(BLOCK)
    for off, n in zip(offsets, sizes):
        used[off + n:off + -(-n // BLOCK) * BLOCK] = 0
    spread = torch.exp(normal(1.0)) * 1e-3 * used
    g, m = normal(1.0) * spread, normal(0.3) * spread
    v = (spread * (1.0 + 0.2 * torch.rand(total, generator=gen, device="cuda"))).square()
    w = normal(0.02)
    for off, n in zip(offsets, sizes):
        w[off + n:off + -(-n // BLOCK) * BLOCK] = 0
    return w, g, m, v


def prepare(case, seed):
    sizes = _sizes(case)
    offsets, total = _layout(sizes)
    op = case["op"]
    w, g, m, v = _values(case, seed)
    state = {"op": op, "case": dict(case), "sizes": sizes, "offsets": offsets, "total": total}
    if op == "norm":
        state["g"] = g.to(DTYPES[case["g"]])
        state["max_norm"] = 0.5 * 1e-3 * math.sqrt(total)
        blocks = torch.tensor([-(-n // BLOCK) for n in sizes], device="cuda")
        state["owner"] = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), blocks)
        state["norms"] = torch.zeros(len(sizes), device="cuda")
    elif op == "load":
        # Moments of a run with 32-bit states, and the empty 8-bit states that take them.
        state["values"] = (m.to(DTYPES[case["values"]]), v.to(DTYPES[case["values"]]))
        state.update(_empty_codes(total))
        state["out"] = tuple(torch.zeros(total, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    elif op == "save":
        state.update(_encode(m, v, None))
        state["out"] = tuple(torch.zeros(total, device="cuda", dtype=DTYPES[case["values"]]) for _ in range(2))
    else:
        state["w"], state["g"] = w.to(DTYPES[case["w"]]), g.to(DTYPES[case["g"]])
        state["master"] = w.clone() if case["master"] else None
        state["scale"] = torch.full((1,), 0.37, device="cuda") if case["clip"] else None
        # Elements of the tensors that decay: they come first.
        large = [i for i, n in enumerate(sizes) if n > MAX_VECTOR]
        state["decayed"] = 0 if not large else (offsets + [total])[large[-1] + 1]
        state["t"] = case["step"] - 1   # steps done before this one
        state["seed"] = int(seed) & 0xFFFFFFFF
        if op == "adamw":
            state["m"], state["v"] = m, v
        else:
            state.update(_encode(m, v, None))
            state["out"] = tuple(torch.zeros(total, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    if own:
        _plan(state)
    return state


def _plan(state):
    """The plan a program keeps beside its tensors."""
    import dimuon_newton_schulz_amd as D
    op, case, sizes, offsets = state["op"], state["case"], state["sizes"], state["offsets"]

    def views(flat, per=1):
        if flat is None:
            return [None] * len(sizes)
        return [flat[o // per:o // per + -(-n // per)] for o, n in zip(offsets, sizes)]

    if op == "norm":
        state["plan"] = D.GradNormPlan(views(state["g"]), max_norm=state["max_norm"], tensor_norms=state["norms"])
        return
    if op in ("save", "load"):
        state["w"] = torch.zeros(state["total"], device="cuda", dtype=torch.bfloat16)
        state["g"] = torch.zeros(state["total"], device="cuda", dtype=torch.bfloat16)
    eight = op != "adamw"
    m_scale, v_scale = (views(state["m_scale"], BLOCK), views(state["v_scale"], BLOCK)) if eight else (views(None),) * 2
    params = [D.AdamWParam(w=wi, g=gi, m=mi, v=vi, m_scale=ms, v_scale=vs, master=ma,
                           weight_decay=DECAY if n > MAX_VECTOR else 0.0)
              for wi, gi, mi, vi, ms, vs, ma, n in zip(
                  views(state["w"]), views(state["g"]), views(state["m"]), views(state["v"]), m_scale, v_scale,
                  views(state.get("master")), sizes)]
    cfg = D.adamw_config_for(params, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                             rounding=case.get("rounding", "nearest"), seed=state.get("seed", 0),
                             grad_scale=state.get("scale"))
    state["plan"] = D.AdamWPlan(params, cfg, step=state.get("t", 0))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        plan = state["plan"]
        if op == "norm":
            return {"norm": plan.run(), "norms": state["norms"]}
        if op == "save":
            m, v = plan.get_state(*state["out"])
            return {"m": m, "v": v}
        if op == "load":
            plan.set_state(*state["values"])
        else:
            plan.step()
        if op == "adamw":
            return _outputs(state, state["m"], state["v"])
        m, v = plan.get_state(*state["out"])
        return _outputs(state, m, v)
    if op == "norm":
        per = torch.zeros(len(state["sizes"]), device="cuda", dtype=torch.float64)
        per.index_add_(0, state["owner"], state["g"].double().square().view(-1, BLOCK).sum(1))
        norm, limit = per.sum().sqrt(), state["max_norm"]
        coef = torch.where(norm <= limit, torch.ones_like(norm), limit / norm)
        return {"norm": torch.stack([norm, coef]).float(), "norms": per.sqrt().float()}
    if op == "save":
        m, v = _decode(state)
        return {"m": m.to(state["out"][0].dtype), "v": v.to(state["out"][1].dtype)}
    if op == "load":
        state.update(_encode(state["values"][0].float(), state["values"][1].float(), None))
        m, v = _decode(state)
        return _outputs(state, m.bfloat16(), v.bfloat16())
    state["t"] += 1
    t = state["t"]
    y = state["g"].float() if state["scale"] is None else state["g"].float() * state["scale"]
    m, v = (state["m"], state["v"]) if op == "adamw" else _decode(state)
    m = BETA1 * m + (1 - BETA1) * y
    v = BETA2 * v + (1 - BETA2) * y * y
    step = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    w = state["w"].float() if state["master"] is None else state["master"]
    step[:state["decayed"]] += DECAY * w[:state["decayed"]]
    w = w - LR * step
    if state["master"] is not None:
        state["master"].copy_(w)
    state["w"].copy_(w)
    if op == "adamw":
        state["m"].copy_(m)
        state["v"].copy_(v)
        return _outputs(state, state["m"], state["v"])
    stochastic = state["case"]["rounding"] == "stochastic"
    state.update(_encode(m, v, _random(state["total"], state["seed"], t) if stochastic else None))
    m, v = _decode(state)
    return _outputs(state, m.bfloat16(), v.bfloat16())


def _outputs(state, m, v):
    out = {"m": m, "v": v}
    if state["op"] in ("adamw", "adamw8"):
        out["w"] = state["w"]
        if state["master"] is not None:
            out["master"] = state["master"]
    return out


# The 8-bit moments.  A block of 256 elements of one tensor shares a float32
# scale.  m: float8 e4m3 times (largest |m| / 256).  v: an unsigned float of
# five exponent and three mantissa bits, the value of code c >= 1 being the
# float32 with the bits (c + 768) << 20, times the block's largest v; code 0
# is zero, and a v above zero has a code of at least 1.
def _empty_codes(total):
    return {"m": torch.zeros(total, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn),
            "v": torch.zeros(total, device="cuda", dtype=torch.uint8),
            "m_scale": torch.zeros(total // BLOCK, device="cuda"),
            "v_scale": torch.zeros(total // BLOCK, device="cuda")}


def _round_bits(x, bits):
    """float32 bits of x plus what is added to the 20 that are dropped."""
    return x.view(torch.int32) + (0x80000 if bits is None else bits * 16 + 8)


def _encode(m, v, random):
    low, high = (None, None) if random is None else (random & 0xFFFF, (random >> 16) & 0xFFFF)
    ms = m.view(-1, BLOCK).abs().amax(1) / 256
    vs = v.view(-1, BLOCK).amax(1)
    ms_all, vs_all = ms.repeat_interleave(BLOCK), vs.repeat_interleave(BLOCK)
    y = torch.where(ms_all > 0, m.abs() / ms_all, 0.0).clamp(max=448.0)
    small = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)   # below 2^-6 the step of e4m3 stays 2^-9
    y = (_round_bits(y + small, low) & -0x100000).view(torch.float32) - small
    y = torch.where(vs_all > 0, v / vs_all, 0.0).clamp(max=1.0), torch.copysign(y, m)
    code = torch.where(v > 0, ((_round_bits(y[0], high) >> 20) - 768).clamp(min=1), 0)
    return {"m": y[1].to(torch.float8_e4m3fn), "v": code.to(torch.uint8), "m_scale": ms, "v_scale": vs}


def _decode(state):
    code = state["v"].int()
    v = torch.where(code > 0, ((code + 768) << 20).view(torch.float32), 0.0)
    return ((state["m"].float().view(-1, BLOCK) * state["m_scale"][:, None]).view(-1),
            (v.view(-1, BLOCK) * state["v_scale"][:, None]).view(-1))


def _mix(x):
    """Mixes the bits of 32-bit integers (held in int32, products wrap)."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * 0x6A09E667
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * (0xBB67AE85 - (1 << 32))
    return x ^ ((x >> 16) & 0xFFFF)


def _mix_int(x):
    x &= 0xFFFFFFFF
    x ^= x >> 16
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x ^= x >> 15
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _key(seed, t, high):
    """Key of the indexes whose upper 32 bits are `high`, for step t."""
    k = _mix_int((t & 0xFFFFFFFF) ^ _mix_int((t >> 32) ^ 0x3C6EF372))
    k = _mix_int((seed & 0xFFFFFFFF) ^ _mix_int((seed >> 32) ^ k))
    return _mix_int(k + high)


def _random(total, seed, t):
    """32 random bits for every flat index (below 2^32 here): m takes the lower 16, v the upper."""
    key = _key(seed, t, 0)
    key = key - (1 << 32) if key >= 1 << 31 else key
    return _mix(torch.arange(total, device="cuda", dtype=torch.int32) + key)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        sq = [s["g"][o:o + n].double().pow(2).sum() for o, n in zip(s["offsets"], s["sizes"])]
        norm = torch.stack(sq).sum().sqrt()
        coef = min(1.0, s["max_norm"] / float(norm))
        return {"norm": torch.tensor([float(norm), coef], dtype=torch.float64), "norms": torch.stack(sq).sqrt()}
    if op == "load":
        m, v = _exact_moments(*(x.double() for x in s["values"]), None)
        return {"m": m, "v": v}
    if op == "adamw":
        m, v = s["m"].double(), s["v"].double()
    else:
        e, f = (s["v"].long() >> 3) - 31, (s["v"].long() & 7).double() / 8
        unit = torch.where(s["v"] == 0, 0.0, torch.ldexp(1 + f, e))
        m = (s["m"].double().view(-1, BLOCK) * s["m_scale"].double()[:, None]).flatten()
        v = (unit.view(-1, BLOCK) * s["v_scale"].double()[:, None]).flatten()
        del e, f, unit
    if op == "save":
        return {"m": m, "v": v}
    t = case["step"]
    y = s["g"].double() * (1.0 if s["scale"] is None else float(s["scale"]))
    m = m.mul_(BETA1).add_((1 - BETA1) * y)
    v = v.mul_(BETA2).add_((1 - BETA2) * y.square())
    del y
    w = (s["w"] if s["master"] is None else s["master"]).double()
    decay = torch.zeros_like(w)
    decay[:s["decayed"]] = DECAY
    w = w - LR * (m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS) + decay * w)
    del decay
    out = {"w": w}
    if s["master"] is not None:
        out["master"] = w
    if op == "adamw8":
        bits = None
        if case["rounding"] == "stochastic":
            bits = (torch.arange(m.numel(), device=m.device) + _key(s["seed"], t, 0)) & 0xFFFFFFFF
            for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85), (16, 1)):
                bits = ((bits ^ (bits >> shift)) * factor) & 0xFFFFFFFF
        m, v = _exact_moments(m, v, bits)
    out.update(m=m, v=v)
    return out


def _exact_moments(m, v, bits):
    """The values that the 8-bit codes of m and v stand for."""
    up = [0.5, 0.5] if bits is None else [((b & 0xFFFF) * 16 + 8).double() / 2 ** 20 for b in (bits, bits >> 16)]
    ms = m.view(-1, BLOCK).abs().amax(1, keepdim=True).expand(-1, BLOCK).flatten() / 256
    y = torch.where(ms > 0, m.abs() / ms, 0.0)
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    m = torch.floor(y / step + up[0]) * step * ms * torch.sign(m)
    del ms
    vs = v.view(-1, BLOCK).amax(1, keepdim=True).expand(-1, BLOCK).flatten()
    y = torch.where(vs > 0, v / vs, 0.0)
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-31).double() - 3)
    q = (torch.floor(y / step + up[1]) * step).clamp(min=1.125 * 2.0 ** -31)
    return m, torch.where(v > 0, q * vs, 0.0)
