"""AdamW (32- and 8-bit moments), the moments as values, and the global
gradient norm: refusals on the CPU, results on the GPU against the float64
oracle.

Bounds count roundings.  U = 2^-24 is half a float32 step relative to the
value.
  m':  beta1, beta1*m, 1-beta1, y = s*g, (1-beta1)*y, sum: at most 6 U of |beta1 m| + |(1-beta1) y|
  v':  two roundings of y count twice through the square; beta2, 1-beta2, two products, sum: 8 U of v'
  w':  numerator and denominator, sqrt and quotient of up to 2 U each: 20 U of the Adam term, plus what the
       error of m' becomes in it; products and sums of the update 4 U; the last sum U of |w'|; the store of a
       bf16 weight half a step, 2^-8 of |w'|.
  8-bit moments: a code may differ from the oracle's only where the unrounded value lies within the float32
       error of a border between two codes; the decoded value is then one code step off.
"""

import ctypes
import os
import sys

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from oracle import adamw_oracle as O

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = [1, 7, 255, 256, 257, 0, 4095, 4096, 4097, 70001]
gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


def announce(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


# ---------------------------------------------------------------------------
# CPU: the oracle's codes and hash, and refusals
# ---------------------------------------------------------------------------
def test_codes_round_trip_and_match_the_fp8_type():
    c = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    got = O.decode_m(c, np.ones(1))
    np.testing.assert_array_equal(got, ref)
    ok = np.isfinite(got)
    np.testing.assert_array_equal(O.encode_m(got[ok], np.ones(1), 0.5), c[ok])
    v = O.decode_v(c[:249], np.ones(1))
    assert v[0] == 0 and v[1] == 1.125 * 2.0 ** -31 and v[248] == 1.0 and (np.diff(v) > 0).all()
    np.testing.assert_array_equal(O.encode_v(v, np.ones(1), 0.5), c[:249])
    # nothing above zero is stored as zero
    assert (O.encode_v(np.array([1e-30, 2.0 ** -33]), np.ones(1), 2.0 ** -17) == 1).all()


def test_hash_is_uniform_and_mixes():
    m, v = O.random_bits(np.arange(1 << 18) + 77 * (1 << 32), seed=0x123456789ABCDEF, t=5)
    n = len(m)
    for r in (m, v):
        x = (r.astype(np.float64) + 0.5) / 65536
        # uniform: mean 1/2 with deviation 1/sqrt(12 n), five of them
        assert abs(x.mean() - 0.5) < 5 / np.sqrt(12 * n)
        assert abs(np.corrcoef(x[1:], x[:-1])[0, 1]) < 5 / np.sqrt(n)
    assert abs(np.corrcoef(m.astype(float), v.astype(float))[0, 1]) < 5 / np.sqrt(n)
    keys = {O.key(s, t) for s in (0, 1, 1 << 32) for t in (1, 2, 1 << 32)}
    assert len(keys) == 9


def fake(count=2, n=1000, block8=False, master=False, base=0x100000000, stride=0x1000000):
    arr = (D.AdamWTensor * count)()
    at = base
    for i in range(count):
        for name in ("w", "g", "m", "v") + (("m_scale", "v_scale") if block8 else ()) + (("master",) if master else ()):
            setattr(arr[i], name, at)
            at += stride
        arr[i].n, arr[i].lr_scale, arr[i].weight_decay = n, 1.0, 0.1
    return arr


def fake_cfg(**kw):
    return D.AdamWConfig(**kw).to_c()


REFUSALS = {
    "null_list": 1, "count0": 1, "n_negative": 1, "n_huge": 6, "pieces": 6, "beta1": 1, "beta_nan": 1, "eps": 1,
    "lr_nan": 1, "w_dtype": 2, "state": 2, "rounding": 1, "null_w": 1, "null_scale": 1, "misaligned_g": 1,
    "misaligned_scale": 1, "lr_scale": 1, "weight_decay": 1, "alias": 4, "alias_scale_in_m": 4, "master_f32": 2,
    "master_some": 1, "grad_scale_misaligned": 1, "grad_scale_in_w": 4, "ws_null": 3, "ws_small": 3,
    "ws_misaligned": 3, "ws_alias": 4, "step0": 1, "step_huge": 1,
}


@built
@pytest.mark.parametrize("kind", sorted(REFUSALS))
def test_adamw_refusals(kind):
    lib = D.load_library()
    block8 = "scale" in kind and not kind.startswith("grad")
    arr, cfg = fake(block8=block8, master=kind.startswith("master")), fake_cfg(state="block8" if block8 else "f32")
    count, ws, ws_bytes, step = 2, 0x700000000000, 1 << 40, 1
    if kind == "null_list":
        arr = None
    elif kind == "count0":
        count = 0
    elif kind == "n_negative":
        arr[1].n = -1
    elif kind == "n_huge":
        arr[1].n = (1 << 40) + 1
    elif kind == "pieces":
        arr = fake(count=9, n=1 << 40)
        count = 9
    elif kind == "beta1":
        cfg.beta1 = 1.0
    elif kind == "beta_nan":
        cfg.beta2 = float("nan")
    elif kind == "eps":
        cfg.eps = -1e-8
    elif kind == "lr_nan":
        cfg.lr = float("nan")
    elif kind == "w_dtype":
        cfg.w_dtype = 7
    elif kind == "state":
        cfg.state = 2
    elif kind == "rounding":
        cfg.rounding = 3
    elif kind == "null_w":
        arr[1].w = None
    elif kind == "null_scale":
        arr[0].v_scale = None
    elif kind == "misaligned_g":
        arr[0].g += 8
    elif kind == "misaligned_scale":
        arr[0].m_scale += 2
    elif kind == "lr_scale":
        arr[1].lr_scale = float("inf")
    elif kind == "weight_decay":
        arr[1].weight_decay = float("nan")
    elif kind == "alias":
        arr[1].w = arr[0].m + 16
    elif kind == "alias_scale_in_m":
        arr[0].m_scale = arr[1].m + 4
    elif kind == "master_f32":
        cfg.w_dtype = 0
    elif kind == "master_some":
        arr[1].master = None
    elif kind == "grad_scale_misaligned":
        cfg.grad_scale = 0x900000000002
    elif kind == "grad_scale_in_w":
        cfg.grad_scale = arr[1].w + 4
    elif kind == "ws_null":
        ws = None
    elif kind == "ws_small":
        ws_bytes = 512
    elif kind == "ws_misaligned":
        ws += 16
    elif kind == "ws_alias":
        ws = arr[0].g
    elif kind == "step0":
        step = 0
    elif kind == "step_huge":
        step = (1 << 62) + 1
    calls = [lambda: lib.adamw_step(arr, count, ctypes.byref(cfg), step, ws, ws_bytes, None)]
    handle = ctypes.c_void_p(0)
    calls.append(lambda: lib.adamw_plan_create(arr, count, ctypes.byref(cfg), step - 1, ws, ws_bytes, None,
                                               ctypes.byref(handle)))
    for call in calls:
        assert call() == REFUSALS[kind], lib.muon_last_error()
        assert lib.muon_last_error() and not handle


@built
def test_null_plans_and_outputs_are_refused():
    lib = D.load_library()
    assert lib.adamw_plan_step(None, None) == 1
    assert lib.adamw_plan_set_lr(None, 1.0, None) == 1
    assert lib.adamw_plan_set_step(None, 1, None) == 1
    assert lib.adamw_plan_get_state(None, 16, 16, 0, None) == 1
    assert lib.adamw_plan_set_state(None, 16, 16, 0, None) == 1
    assert lib.muon_grad_norm_plan_run(None, None) == 1
    lib.adamw_plan_destroy(None)
    lib.muon_grad_norm_plan_destroy(None)
    cfg = fake_cfg()
    assert lib.adamw_workspace_bytes(fake(), 2, ctypes.byref(cfg), None) == 1
    assert lib.adamw_workspace_bytes(fake(), 2, None, ctypes.byref(ctypes.c_size_t())) == 1
    assert lib.muon_status_string(7)


@built
def test_state_elems_and_workspace():
    lib, out, nbytes = D.load_library(), ctypes.c_int64(0), ctypes.c_size_t(0)
    arr = fake(3)
    arr[0].n, arr[1].n, arr[2].n = 1, 0, 257
    assert lib.adamw_state_elems(arr, 3, ctypes.byref(out)) == 0 and out.value == 256 + 512
    assert lib.adamw_workspace_bytes(arr, 3, ctypes.byref(fake_cfg()), ctypes.byref(nbytes)) == 0
    assert 0 < nbytes.value < 8192   # counters (33 lines of 128 bytes), three descriptors, two units
    # gradients may share memory: the NULL workspace is what is refused
    arr = fake(2)
    arr[1].g = arr[0].g
    assert lib.adamw_step(arr, 2, ctypes.byref(fake_cfg()), 1, None, 0, None) == 3
    # empty tensors' pointers are not looked at
    arr[0].n, arr[0].w = 0, None
    assert lib.adamw_step(arr, 2, ctypes.byref(fake_cfg()), 1, None, 0, None) == 3


def fake_grads(sizes=(1000, 2000)):
    arr = (D.MuonGrad * len(sizes))()
    for i, n in enumerate(sizes):
        arr[i].g, arr[i].n, arr[i].dtype = 0x100000000 + i * 0x1000000, n, i % 2
    return arr


@built
@pytest.mark.parametrize("kind,want", [("null", 1), ("count0", 1), ("dtype", 2), ("n", 1), ("null_g", 1),
                                       ("misaligned", 1), ("max_zero", 1), ("max_nan", 1), ("out_null", 1),
                                       ("out_misaligned", 1), ("out_in_g", 4), ("norms_in_out", 4), ("ws_null", 3),
                                       ("ws_small", 3), ("ws_alias", 4)])
def test_grad_norm_refusals(kind, want):
    lib = D.load_library()
    arr, count, limit, out, norms = fake_grads(), 2, 1.0, 0x200000000, 0x300000000
    ws, ws_bytes = 0x700000000000, 1 << 30
    if kind == "null":
        arr = None
    elif kind == "count0":
        count = 0
    elif kind == "dtype":
        arr[0].dtype = 2
    elif kind == "n":
        arr[0].n = -5
    elif kind == "null_g":
        arr[1].g = None
    elif kind == "misaligned":
        arr[1].g += 4
    elif kind == "max_zero":
        limit = 0.0
    elif kind == "max_nan":
        limit = float("nan")
    elif kind == "out_null":
        out = None
    elif kind == "out_misaligned":
        out += 2
    elif kind == "out_in_g":
        out = arr[0].g + 8
    elif kind == "norms_in_out":
        norms = out + 4
    elif kind == "ws_null":
        ws = None
    elif kind == "ws_small":
        ws_bytes = 256
    elif kind == "ws_alias":
        ws = arr[1].g
    handle = ctypes.c_void_p(0)
    assert lib.muon_grad_norm(arr, count, limit, out, norms, ws, ws_bytes, None) == want, lib.muon_last_error()
    assert lib.muon_grad_norm_plan_create(arr, count, limit, out, norms, ws, ws_bytes, None,
                                          ctypes.byref(handle)) == want
    assert not handle and lib.muon_last_error()


@built
def test_muon_refuses_a_grad_scale_it_would_overwrite():
    lib = D.load_library()
    arr = (D.MuonMatrix * 1)()
    arr[0].w, arr[0].g, arr[0].mom, arr[0].m, arr[0].n = 0x100000000, 0x110000000, 0x120000000, 64, 256
    cfg, _ = D.StepConfig().to_c()
    for ptr, want in ((0x900000000002, 1), (arr[0].w + 4, 4), (0x700000000100, 4), (0x900000000000, 3)):
        cfg.grad_scale = ptr
        ws = 0x700000000000 if want != 3 else None
        assert lib.muon_step(arr, 1, ctypes.byref(cfg), ws, 1 << 40, None) == want, lib.muon_last_error()


@built
def test_python_checks():
    w = torch.zeros(300, dtype=torch.bfloat16)
    p = D.adamw_param(w, w.clone(), state="block8", master=True)
    assert p.m.dtype == torch.float8_e4m3fn and p.v.dtype == torch.uint8 and p.m_scale.numel() == 2
    assert p.master.dtype == torch.float32
    with pytest.raises(ValueError):
        D.adamw_param(w, w, state="4bit")
    cfg = D.adamw_config_for([p])
    assert cfg.state == "block8" and cfg.w_dtype == "bf16"

    def refused(**kw):
        q = D.AdamWParam(**{**p.__dict__, **kw})
        with pytest.raises(ValueError):
            D._marshal_adamw([q], cfg)

    D._marshal_adamw([p], cfg)
    refused(m=p.m.view(torch.uint8))
    refused(v=torch.zeros(300))
    refused(m_scale=None)
    refused(m_scale=torch.zeros(3))
    refused(g=torch.zeros(300))
    refused(g=torch.zeros(301, dtype=torch.bfloat16))
    refused(w=torch.zeros(600, dtype=torch.bfloat16)[::2])
    refused(master=torch.zeros(300, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        D.AdamWConfig(grad_scale=torch.zeros(1)).to_c()       # not on the GPU
    for call in (lambda: D.adamw_step([p], cfg, 1), lambda: D.AdamWPlan([p], cfg), lambda: D.grad_norm([w]),
                 lambda: D.GradNormPlan([w]), lambda: D.grad_norm([])):
        with pytest.raises(ValueError):   # tensors in host memory, no tensors
            call()
    with pytest.raises(ValueError):
        D._marshal_grads([torch.zeros(3, dtype=torch.float64)], None, None)


# ---------------------------------------------------------------------------
# GPU: one step against the oracle
# ---------------------------------------------------------------------------
def tensors(sizes, w, g, state, master, seed=0, std=1e-3):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        spread = torch.exp(torch.randn(n, generator=gen)) * std
        wi = (torch.randn(n, generator=gen) * 0.02).to(DT[w]).cuda()
        gi = (torch.randn(n, generator=gen) * spread).to(DT[g]).cuda()
        out.append(D.adamw_param(wi, gi, state=state, master=master, lr_scale=1.0 + 0.25 * (i % 3),
                                 weight_decay=0.1 * (i % 2)))
    return out


def host(t):
    return t.detach().double().cpu().numpy().ravel() if t.dtype != torch.float8_e4m3fn else \
        t.view(torch.uint8).cpu().numpy().ravel()


def snapshot(p):
    s = {k: host(getattr(p, k)) for k in ("w", "g", "m", "v", "m_scale", "v_scale", "master")
         if getattr(p, k) is not None}
    if "m_scale" in s:
        s["m_codes"], s["v_codes"] = s["m"], s["v"]
        s["m"], s["v"] = O.decode_m(s["m"], s["m_scale"]), O.decode_v(s["v"], s["v_scale"])
    return s


def check_codes(code, want, pos, up, err_pos, ctx):
    """Codes equal the oracle's, but within err_pos code steps of a border.
    (m's codes 0x00 and 0x80 both stand for zero: where |m| is below its own
    float32 error, its sign is not determined.)"""
    zero = lambda c: np.where((c == 0x80) & (ctx[-1] == "m"), 0, c)   # noqa: E731
    off = np.flatnonzero(zero(code) != zero(want))
    if len(off):
        x = pos[off] + (up[off] if np.ndim(up) else up)
        dist = np.abs(x - np.rint(x))
        assert (dist <= err_pos[off]).all(), (ctx, off[:5], code[off][:5], want[off][:5], dist[:5], err_pos[off][:5])


def check_step(before, after, cfg, p, t, first, scale, ctx):
    b1, b2 = cfg.beta1, cfg.beta2
    m, v = O.moments(before["m"], before["v"], before["g"], b1, b2, scale)
    em = 6 * U * (np.abs(b1 * before["m"]) + np.abs((1 - b1) * before["g"] * scale)) + 1e-45
    ev = 8 * U * np.abs(v) + 1e-45
    w0 = before.get("master", before["w"])
    w1 = O.update(w0, m, v, t, cfg.lr, b1, b2, cfg.eps, p.lr_scale, p.weight_decay)
    adam = np.abs(w1 - w0 * (1 - cfg.lr * p.weight_decay))
    den = np.sqrt(v / (1 - b2 ** t)) + cfg.eps
    ew = 20 * U * adam + abs(cfg.lr * p.lr_scale) * em / (1 - b1 ** t) / den + \
        4 * U * (adam + abs(cfg.lr * p.weight_decay) * np.abs(w0)) + U * np.abs(w1)
    if "master" in before:
        assert (np.abs(after["master"] - w1) <= ew).all(), ctx
        w1, ew = after["master"], 0.0
    if p.w.dtype == torch.bfloat16:
        ew = ew + 2.0 ** -8 * np.abs(w1)
    worst = np.abs(after["w"] - w1) - ew
    assert (worst <= 0).all(), (ctx, "w", worst.max())
    if cfg.state == "f32":
        assert (np.abs(after["m"] - m) <= em).all(), (ctx, "m")
        assert (np.abs(after["v"] - v) <= ev).all(), (ctx, "v")
        return
    if not len(m):
        return
    ms, vs = O.scales(m, v)
    peak = np.array([np.max(b) for b in O._blocks(em)])
    assert (np.abs(after["m_scale"] - ms) <= peak / 256 + U * ms).all(), (ctx, "m_scale")
    assert (np.abs(after["v_scale"] - vs) <= 9 * U * vs).all(), (ctx, "v_scale")
    if cfg.rounding == "nearest":
        um = uv = 0.5
    else:
        bits = O.random_bits(first + np.arange(len(m)), cfg.seed, t)
        um, uv = [(b.astype(np.float64) * 16 + 8) / 2 ** 20 for b in bits]
    # Positions are |x| / (scale step): the errors of x, of the scale and of the quotient, then of the sum with
    # 2^-6 below the normal range (half a float32 step of at most 2^-5: 2^-29 of values whose step is 2^-9).
    sm, sv = O._spread(after["m_scale"], len(m)), O._spread(after["v_scale"], len(m))
    pos, step = O.positions(m, after["m_scale"], -6)
    with np.errstate(divide="ignore", invalid="ignore"):
        err = np.where(sm > 0, (em + 4 * U * np.abs(m)) / (sm * step), 0.0) + 2.0 ** -20
    check_codes(after["m_codes"], O.encode_m(m, after["m_scale"], um), pos, um, err, (ctx, "m"))
    pos, step = O.positions(v, after["v_scale"], -31)
    with np.errstate(divide="ignore", invalid="ignore"):
        err = np.where(sv > 0, (ev + 4 * U * v) / (sv * step), 0.0) + 1e-12
    check_codes(after["v_codes"], O.encode_v(v, after["v_scale"], uv), pos, uv, err, (ctx, "v"))


FORMS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "f32", False), ("bf16", "bf16", False),
         ("bf16", "bf16", True), ("bf16", "f32", True)]
STATES = [("f32", "nearest"), ("block8", "nearest"), ("block8", "stochastic")]


@gpu
@pytest.mark.parametrize("state,rounding", STATES)
@pytest.mark.parametrize("w,g,master", FORMS)
def test_steps_match_the_oracle(w, g, master, state, rounding):
    announce(f"adamw {w}/{g} master={master} {state} {rounding}")
    ps = tensors(SIZES, w, g, state, master, seed=3)
    scale = torch.tensor([0.37], device="cuda")
    cfg = D.adamw_config_for(ps, lr=3e-3, eps=1e-8, rounding=rounding, seed=0xABCDEF0123456789, grad_scale=scale)
    plan = D.AdamWPlan(ps, cfg, step=0)
    offsets = plan.state_offsets()
    for t in range(1, 4):
        before = [snapshot(p) for p in ps]
        plan.step()
        after = [snapshot(p) for p in ps]
        for i, p in enumerate(ps):
            check_step(before[i], after[i], cfg, p, t, offsets[i], float(scale), f"tensor {i} step {t}")
        for i, p in enumerate(ps):   # another gradient for the next step
            p.g.copy_(-0.7 * p.g.roll(1))


@gpu
@pytest.mark.parametrize("state,rounding", STATES)
def test_stateless_step_equals_the_plan(state, rounding):
    announce(f"adamw stateless {state} {rounding}")
    a, b = (tensors(SIZES, "bf16", "bf16", state, True, seed=5) for _ in range(2))
    cfg = [D.adamw_config_for(x, rounding=rounding, seed=7) for x in (a, b)]
    plan = D.AdamWPlan(a, cfg[0], step=11)
    ws = None
    for t in (12, 13):
        plan.step()
        ws = D.adamw_step(b, cfg[1], t, workspace=ws)
        for p, q in zip(a, b):
            for name in ("w", "m", "v", "m_scale", "v_scale", "master"):
                x, y = getattr(p, name), getattr(q, name)
                if x is not None and x.numel():
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (t, name)


@gpu
@pytest.mark.parametrize("state", ["f32", "block8"])
def test_a_step_touches_nothing_behind_its_tensors(state):
    """Odd sizes inside larger buffers: what follows every tensor stays."""
    announce(f"adamw guards {state}")
    n = 1023
    for w in ("f32", "bf16"):
        def guarded(m, dtype):
            t = torch.full((m + 64,), 77, device="cuda").to(dtype)
            t[:m] = 0
            return t
        bufs = {"w": guarded(n, DT[w]), "g": guarded(n, DT[w]), "m": guarded(n, torch.uint8 if state == "block8" else torch.float32),
                "v": guarded(n, torch.uint8 if state == "block8" else torch.float32)}
        if state == "block8":
            bufs["m_scale"], bufs["v_scale"] = guarded(4, torch.float32), guarded(4, torch.float32)
        bufs["g"][:n] = 0.5
        view = {k: t[:4] if k.endswith("scale") else t[:n] for k, t in bufs.items()}
        if state == "block8":
            view["m"] = view["m"].view(torch.float8_e4m3fn)
        p = D.AdamWParam(**view)
        plan = D.AdamWPlan([p], D.adamw_config_for([p]))
        plan.step()
        m, v = (torch.full((plan.state_elems,), 5.0, device="cuda") for _ in range(2))
        plan.get_state(m, v)
        plan.set_state(m, v)
        for k, t in bufs.items():
            size = 4 if k.endswith("scale") else n
            assert (t[size:].float() == 77).all(), k
        assert (m[n:] == 5).all() and (v[n:] == 5).all()
        assert (view["w"].float() != 0).all()


@gpu
@pytest.mark.parametrize("state,rounding", STATES)
def test_edge_values(state, rounding):
    """Zero gradients, one-sided huge and tiny values, NaN and Inf: only the
    elements that hold them, and no other element of their block, are lost."""
    announce(f"adamw edge values {state} {rounding}")
    n = 256 * 6 + 10
    g = torch.zeros(n)
    g[256:512] = torch.randn(256, generator=torch.Generator().manual_seed(1)) * 1e-3
    g[300], g[301], g[302] = float("nan"), float("inf"), -float("inf")
    g[512:768] = 1e-22          # squares are denormal or zero
    g[768:1024] = 1e15
    g[800] = 1e-15
    g[1024] = 1.0               # one element of an otherwise untouched block
    g[1536:] = 1e-4
    p = D.adamw_param(torch.ones(n, device="cuda"), g.cuda(), state=state, weight_decay=0.1)
    cfg = D.adamw_config_for([p], lr=0.01, rounding=rounding, seed=3)
    plan = D.AdamWPlan([p], cfg)
    plan.step()
    plan.step()
    m, v = (x.cpu() for x in plan.get_state())
    w = p.w.cpu()
    lost = torch.zeros(n, dtype=torch.bool)
    lost[300:303] = True
    assert torch.isfinite(w[~lost]).all() and not torch.isfinite(w[lost]).any()
    assert torch.isfinite(m[:n][~lost]).all() and torch.isfinite(v[:n][~lost]).all()
    assert not torch.isfinite(m[:n][lost]).any()
    keep = 1 - 0.01 * 0.1
    zero = (g == 0) & ~lost
    assert (m[:n][zero] == 0).all() and (v[:n][zero] == 0).all()
    # Two decays of a weight without gradients: two products of two roundings each.
    assert (w[zero] - keep ** 2).abs().max() <= 8 * U
    # A constant gradient far above eps moves a weight by lr a step: 8-bit moments of a block of equal values are exact.
    assert (w[801:1024] - (keep * (keep - 0.01) - 0.01)).abs().max() <= 60 * U
    assert v[800] > 0
    # The small element of a block of large ones: its denominator is at least its own v, so the step is at most lr.
    assert keep ** 2 - 2 * 0.01 * 1.0001 <= w[800] <= keep ** 2 + 1e-6


@gpu
def test_eps_zero_and_tiny_gradients():
    """eps = 0: a weight moves by lr for any gradient whose square float32 holds as a normal number."""
    announce("adamw eps 0")
    g = torch.tensor([1e-15, -1e-10, 1.0, 1e10, -1e18], device="cuda")
    p = D.adamw_param(torch.zeros(5, device="cuda"), g)
    D.adamw_step([p], D.adamw_config_for([p], lr=0.5, eps=0.0), 1)
    np.testing.assert_allclose(host(p.w), -0.5 * np.sign(host(g)), rtol=40 * U)


@gpu
def test_stochastic_rounding_is_unbiased():
    """v of a constant gradient under many seeds: the mean code value is the unrounded one."""
    announce("adamw stochastic rounding mean")
    n, reps = 256 * 64, 64
    base = torch.rand(n, generator=torch.Generator().manual_seed(2)) * 0.9 + 0.1
    base[::256] = 1.0
    total, exact = 0.0, None
    for seed in range(reps):
        p = D.adamw_param(torch.zeros(n, device="cuda"), base.cuda(), state="block8")
        plan = D.AdamWPlan([p], D.adamw_config_for([p], seed=seed, beta1=0.0, beta2=0.0))
        plan.step()
        m, v = plan.get_state()
        total = total + torch.stack([m, v]).double().cpu()
    exact = torch.stack([base.double(), base.double().square()])
    # A rounding to steps of at most 1/8 of the value has a variance of at most (1/16)^2 of its square; the mean over
    # all elements and seeds lies within five of its deviations.
    mean = ((total / reps / exact) - 1).mean(1)
    assert mean.abs().max() < 5 * (1 / 16) / np.sqrt(n * reps)


# ---------------------------------------------------------------------------
# GPU: values of the moments
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("state", ["f32", "block8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_values(state, dtype):
    announce(f"adamw state values {state} {dtype}")
    ps = tensors(SIZES, "f32", "f32", state, False, seed=9)
    plan = D.AdamWPlan(ps, D.adamw_config_for(ps, seed=1))
    offs = plan.state_offsets()
    gen = torch.Generator().manual_seed(4)
    spread = torch.exp(3 * torch.randn(plan.state_elems, generator=gen))
    m = (torch.randn(plan.state_elems, generator=gen) * spread).to(DT[dtype]).cuda()
    v = spread.square().to(DT[dtype]).cuda()
    v[: 128] = 0
    m[: 64] = 0
    plan.set_state(m, v)
    for o, p in zip(offs, ps):
        n = p.w.numel()
        if n == 0:
            continue
        mi, vi = host(m[o:o + n]), host(v[o:o + n])
        s = snapshot(p)
        if state == "f32":
            np.testing.assert_array_equal(s["m"], mi)
            np.testing.assert_array_equal(s["v"], vi)
        else:
            ms, vs = O.scales(mi, vi)
            np.testing.assert_array_equal(s["m_scale"], ms)
            np.testing.assert_array_equal(s["v_scale"], vs)
            # nearest: one quotient's rounding (2 U of the position) decides only next to a border
            pos, _ = O.positions(mi, ms, -6)
            check_codes(s["m_codes"], O.encode_m(mi, ms, 0.5), pos, 0.5, 4 * U * pos + 2.0 ** -20, (n, "m"))
            pos, _ = O.positions(vi, vs, -31)
            check_codes(s["v_codes"], O.encode_v(vi, vs, 0.5), pos, 0.5, 4 * U * pos, (n, "v"))
    got = plan.get_state(dtype=DT[dtype])
    half = U if dtype == "f32" else 2.0 ** -8
    for o, p in zip(offs, ps):
        n, s = p.w.numel(), snapshot(p)
        for k, name in enumerate(("m", "v")):
            x = host(got[k][o:o + n])
            assert (np.abs(x - s[name]) <= 1.01 * half * np.abs(s[name]) + U * np.abs(s[name])).all(), name
    # Float32 values of 8-bit moments give the same codes again.
    codes = [snapshot(p) for p in ps]
    plan.set_state(*plan.get_state())
    for s, p in zip(codes, ps):
        for k, x in snapshot(p).items():
            np.testing.assert_array_equal(x, s[k], err_msg=k)


@gpu
def test_loading_rounds_halfway_values_up():
    """Every pair of bf16 mantissas as a block's largest value and an element:
    quotients halfway between two codes, and next to halfway, at several
    magnitudes.  Quotients of 8-bit mantissas that are not halfway differ from
    it by 2^-16 of their value at least, so float32 quotients decide them all."""
    announce("adamw halfway values")
    mant = 1 + np.arange(128) / 128
    for exp in (-60, -3, 0, 20):
        # One block per largest value: 127 elements below it, from each of two binades.
        rows = []
        for top in mant:
            below = np.concatenate([mant[mant < top], mant / 2, [0.0] * 128])[:255]
            rows.append(np.concatenate([[top], below]))
        x = np.ldexp(np.concatenate(rows), exp)
        m = torch.from_numpy(np.where(np.arange(len(x)) % 3 == 0, -x, x)).to(torch.bfloat16).cuda()
        v = torch.from_numpy(x).to(torch.bfloat16).cuda()
        assert np.array_equal(host(v), x)
        p = D.adamw_param(torch.zeros(len(x), device="cuda"), torch.zeros(len(x), device="cuda"), state="block8")
        D.AdamWPlan([p], D.adamw_config_for([p])).set_state(m, v)
        ms, vs = O.scales(host(m), host(v))
        np.testing.assert_array_equal(host(p.m_scale), ms)
        np.testing.assert_array_equal(host(p.m), O.encode_m(host(m), ms, 0.5))
        np.testing.assert_array_equal(host(p.v), O.encode_v(host(v), vs, 0.5))


@gpu
def test_moving_between_32_and_8_bits():
    """A run with 32-bit moments goes on with 8-bit ones: every value within half a code step."""
    announce("adamw 32 to 8 bits")
    a = tensors(SIZES, "f32", "f32", "f32", False, seed=12)
    plan = D.AdamWPlan(a, D.adamw_config_for(a))
    plan.step()
    m, v = plan.get_state()
    b = [D.adamw_param(p.w, p.g, state="block8") for p in a]
    other = D.AdamWPlan(b, D.adamw_config_for(b), step=1)
    other.set_state(m, v)
    m8, v8 = other.get_state()
    for o, p in zip(plan.state_offsets(), a):
        n = p.w.numel()
        if n == 0:
            continue
        x, y = host(m[o:o + n]), host(v[o:o + n])
        ms, vs = O.scales(x, y)
        step = O.positions(x, ms, -6)[1] * O._spread(ms, n)
        assert (np.abs(host(m8[o:o + n]) - x) <= step * (0.5 + 1e-5)).all()
        step = O.positions(y, vs, -31)[1] * O._spread(vs, n)
        assert (np.abs(host(v8[o:o + n]) - y) <= step * (0.5 + 1e-5) + 2.0 ** -30 * O._spread(vs, n)).all()


@gpu
def test_state_value_buffers_are_checked():
    announce("adamw state value refusals")
    ps = tensors([1000], "f32", "f32", "block8", False)
    plan = D.AdamWPlan(ps, D.adamw_config_for(ps))
    ok = torch.zeros(plan.state_elems, device="cuda")
    for bad in (torch.zeros(1000, device="cuda"), ok.double(), ok.cpu()):
        with pytest.raises(ValueError):
            plan.get_state(bad, ok)
    with pytest.raises(ValueError):
        plan.get_state(ok)
    with pytest.raises(D.MuonError) as e:
        plan.get_state(ok, ok)
    assert e.value.status == 4
    w = torch.zeros(plan.state_elems * 2, device="cuda")
    q = D.adamw_param(w[:1000], ps[0].g)
    other = D.AdamWPlan([q], D.adamw_config_for([q]))
    with pytest.raises(D.MuonError) as e:
        other.set_state(w[:other.state_elems], ok)
    assert e.value.status == 4


# ---------------------------------------------------------------------------
# GPU: gradient norm
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("sizes", [[1], [0], [0, 5, 0], [7, 4096, 4097, 1, 0, 250001], [3] * 5000,
                                   [9_000_001, 17, 2_000_003, 40, 8192 * 3]])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_grad_norm(sizes, kind):
    announce(f"grad norm {len(sizes)} tensors {kind}")
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    grads = [torch.randn(n, generator=gen, device="cuda").to(
        DT[kind] if kind in DT else (torch.float32, torch.bfloat16)[i % 2]) for i, n in enumerate(sizes)]
    for limit in (float("inf"), 0.5):
        norms = torch.full((len(sizes),), -1.0, device="cuda")
        norm, coef, each = O.grad_norm([host(g) for g in grads], limit)
        plan = D.GradNormPlan(grads, limit, tensor_norms=norms)
        for _ in range(2):   # the second run finds the first's ticket and sums
            got = host(plan.run())
            # binary64 sums: their error is far below the float32 store's half step
            assert abs(got[0] - norm) <= 1.01 * U * norm and abs(got[1] - coef) <= 1.01 * U * coef
            assert (np.abs(host(norms) - each) <= 1.01 * U * each).all()
        again = D.grad_norm(grads, limit)
        assert torch.equal(again, plan.out)


@gpu
def test_grad_norm_extremes():
    announce("grad norm extremes")
    big = torch.full((1000,), 1e30, device="cuda")
    out = host(D.grad_norm([big], 1.0))
    assert abs(out[0] / (float(big[0]) * np.sqrt(1000)) - 1) < 3 * U and abs(out[1] * out[0] - 1) < 3 * U
    tiny = torch.full((10,), 1e-30, device="cuda")
    assert abs(host(D.grad_norm([tiny]))[0] / (float(tiny[0]) * np.sqrt(10)) - 1) < 3 * U
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.ones(70000, device="cuda")
        x[69999] = bad
        y = torch.ones(10, device="cuda")
        norms = torch.zeros(2, device="cuda")
        out = D.grad_norm([x, y], 1.0, tensor_norms=norms)
        if bad != bad:
            assert out.isnan().all()
        else:
            assert out[0] == float("inf") and out[1] == 0
        assert not torch.isfinite(norms[0]) and abs(float(norms[1]) - 10 ** 0.5) < 1e-6
    # equal to the limit: not clipped
    assert D.grad_norm([torch.full((4,), 0.5, device="cuda")], 1.0).tolist() == [1.0, 1.0]


# ---------------------------------------------------------------------------
# GPU: streams, graphs, and the operators together
# ---------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("state", ["f32", "block8"])
def test_steps_repeat_on_another_stream_and_captured(state):
    announce(f"adamw streams and graphs {state}")
    sets = [tensors(SIZES, "bf16", "bf16", state, True, seed=21) for _ in range(3)]
    cfgs = [D.adamw_config_for(s, seed=5) for s in sets]
    plans = [D.AdamWPlan(s, c, step=3) for s, c in zip(sets, cfgs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plans[2].step()

    def same(ctx):
        torch.cuda.synchronize()
        for p, q, r in zip(*sets):
            for name in ("w", "m", "v", "m_scale", "v_scale", "master"):
                x, y, z = (getattr(s, name) for s in (p, q, r))
                if x is not None and x.numel():
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (ctx, "stream", name)
                    assert torch.equal(x.view(torch.uint8), z.view(torch.uint8)), (ctx, "graph", name)

    for k in range(4):
        plans[0].step()
        plans[1].step(side)
        graph.replay()
        same(k)
        if k == 1:
            for i, p in enumerate(plans):
                p.set_lr(2e-4, side if i == 1 else None)
        if k == 2:
            for i, p in enumerate(plans):
                p.set_step(100, side if i == 1 else None)
    ws, other = plans[0].workspace.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):   # an upload cannot be captured: refused, and the capture goes on
        with pytest.raises(D.MuonError) as e:
            D.adamw_step(sets[0], cfgs[0], 1, workspace=ws)
        plans[0].step()
    assert e.value.status == 6


@gpu
def test_one_plan_in_two_graphs_and_eager_steps_between():
    """Two captured graphs of one plan share its workspace: replays of either,
    with eager steps between them, are the next steps."""
    announce("adamw two graphs of one plan")
    a, b = (tensors(SIZES + [300000], "bf16", "f32", "block8", False, seed=41) for _ in range(2))
    plans = [D.AdamWPlan(x, D.adamw_config_for(x, seed=9)) for x in (a, b)]
    norms = [D.GradNormPlan([p.g for p in x], 1e-3) for x in (a, b)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for g in graphs:
        with torch.cuda.graph(g):
            norms[1].run()
            plans[1].step()
    for how in (0, 1, 1, "eager", 0, "eager", 1, 0):
        norms[0].run()
        plans[0].step()
        if how == "eager":
            norms[1].run()
            plans[1].step()
        else:
            graphs[how].replay()
        torch.cuda.synchronize()
        assert torch.equal(norms[0].out, norms[1].out)
        for p, q in zip(a, b):
            for name in ("w", "m", "v", "m_scale", "v_scale"):
                x, y = getattr(p, name), getattr(q, name)
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)) if x.numel() else True, (how, name)


@gpu
@pytest.mark.parametrize("variant", ["muon", "dimuon"])
@pytest.mark.parametrize("nesterov", [False, True])
def test_grad_scale_in_muon_equals_scaled_gradients(variant, nesterov):
    """s * G in the step equals a step over gradients scaled beforehand, bit
    for bit; s = 1 equals a step without a scale."""
    announce(f"{variant} grad_scale nesterov={nesterov}")
    shapes = [(8, 1000), (1000, 8), (33, 500), (200, 300), (300, 200)]
    for ns in ("bf16", "f32"):
        results = {}
        for how in ("none", "one", "scaled", "pre"):
            gen = torch.Generator(device="cuda").manual_seed(8)
            ps = []
            for s in shapes:
                w, g, m = (torch.randn(s, generator=gen, device="cuda") for _ in range(3))
                ps.append(D.Param(w=w, g=g * 0.37 if how == "pre" else g, mom=m))
            scale = {"one": 1.0, "scaled": 0.37}.get(how)
            cfg = D.config_for(ps, ns_dtype=ns, nesterov=nesterov,
                               grad_scale=None if scale is None else torch.tensor([scale], device="cuda"))
            plan = D.Plan(ps, cfg, dimuon=variant == "dimuon")
            plan.step()
            plan.step()
            results[how] = [(p.w, p.mom) for p in ps]
        for a, b in (("none", "one"), ("pre", "scaled")):
            for i, (x, y) in enumerate(zip(results[a], results[b])):
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]), (ns, a, b, shapes[i])


@gpu
def test_a_training_step_of_both_optimizers_under_one_clip():
    """One global norm over all gradients; Muon takes the matrices, AdamW the
    rest; eager and captured steps agree, and AdamW's part meets the oracle."""
    announce("clip + muon + adamw")
    runs = []
    for _ in range(2):
        gen = torch.Generator(device="cuda").manual_seed(30)
        mats = [D.Param(*(torch.randn(s, generator=gen, device="cuda").bfloat16() for _ in range(3)))
                for s in [(8, 512), (256, 384), (384, 256)]]
        rest = tensors([5000, 384, 384], "bf16", "bf16", "block8", True, seed=31, std=1.0)
        out = torch.zeros(2, device="cuda")
        norm = D.GradNormPlan([p.g for p in mats] + [p.g for p in rest], max_norm=1.0, out=out)
        muon = D.Plan(mats, D.config_for(mats, grad_scale=out[1:]), dimuon=False)
        adam = D.AdamWPlan(rest, D.adamw_config_for(rest, grad_scale=out[1:], seed=2))
        runs.append((mats, rest, norm, muon, adam, out))

    def step(r):
        r[2].run()
        r[3].step()
        r[4].step()

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(runs[1])
    for t in range(1, 4):
        before = [snapshot(p) for p in runs[0][1]]
        step(runs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(runs[0][5], runs[1][5])
        want = O.grad_norm([host(p.g) for p in runs[0][0] + runs[0][1]], 1.0)
        got = host(runs[0][5])
        assert abs(got[0] - want[0]) <= 1.01 * U * want[0] and abs(got[1] - want[1]) <= 1.01 * U
        for a, b in zip(runs[0][0], runs[1][0]):
            assert torch.equal(a.w, b.w) and torch.equal(a.mom, b.mom)
        offs = runs[0][4].state_offsets()
        for i, (p, q) in enumerate(zip(runs[0][1], runs[1][1])):
            check_step(before[i], snapshot(p), runs[0][4].cfg, p, t, offs[i], got[1], f"tensor {i} step {t}")
            assert torch.equal(p.w, q.w) and torch.equal(p.master, q.master) and torch.equal(p.v, q.v)
        for r in runs:
            for p in r[0] + r[1]:
                p.g.mul_(-0.5)


@gpu
def test_batches_without_elements():
    announce("empty batches")
    e = torch.zeros(0, device="cuda")
    for state in ("f32", "block8"):
        ps = [D.adamw_param(e, e, state=state) for _ in range(3)]
        plan = D.AdamWPlan(ps, D.adamw_config_for(ps))
        for _ in range(3):
            plan.step()
        m, v = plan.get_state()
        plan.set_state(m, v)
        assert m.numel() == v.numel() == 0
        D.adamw_step(ps, D.adamw_config_for(ps), 1)
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("state", ["f32", "block8"])
def test_many_steps_and_many_small_tensors(state):
    """200 steps of 300 tensors: the step number that the device counts is the
    one the bias corrections need (a weight with a constant gradient moves by
    lr a step)."""
    announce(f"adamw many steps {state}")
    ps = [D.adamw_param(torch.zeros(n, device="cuda"), torch.full((n,), 0.01 * (n % 5 + 1), device="cuda"), state=state)
          for n in range(1, 301)]
    plan = D.AdamWPlan(ps, D.adamw_config_for(ps, lr=1e-3, eps=0.0, seed=3))
    for _ in range(200):
        plan.step()
    for p in ps:
        # Equal values of a block are stored exactly but for float32 roundings, which the moments' ratio keeps over
        # 200 steps within 200 times the 20 U of one.
        w = host(p.w)
        assert (np.abs(w + 0.2) <= 0.2 * 200 * 20 * U).all(), w


@gpu
def test_launch_hook_names_the_new_launches():
    announce("launch hook")
    ps = tensors([1000], "f32", "f32", "block8", False)
    plan = D.AdamWPlan(ps, D.adamw_config_for(ps))
    norm = D.GradNormPlan([ps[0].g])
    m, v = plan.get_state()
    with D.LaunchTimer(8) as t:
        for call, kind in ((plan.step, "adamw"), (lambda: plan.get_state(m, v), "state_get"),
                           (lambda: plan.set_state(m, v), "state_set"), (norm.run, "grad_norm")):
            call()
            torch.cuda.synchronize()
            assert t.recorded() == 2
            (got, ms), = t.durations(2)
            assert got == kind and ms >= 0


@gpu
def test_offsets_beyond_32_bits():
    """A tensor of more than 2^32 elements: its last elements against the oracle, and its norm."""
    n = (1 << 32) + 300
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of device memory")
    announce(f"adamw {n} elements")
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-700:] = (torch.arange(700, device="cuda") - 350) * 1e-3
    g[5] = 0.25
    p = D.adamw_param(w, g, state="block8")
    cfg = D.adamw_config_for([p], seed=77)
    plan = D.AdamWPlan([p], cfg)
    first = n - n % 256 - 512
    tail = slice(first, n)

    def view():
        s = {"w": host(w[tail]), "g": host(g[tail]), "m_codes": host(p.m[tail]), "v_codes": host(p.v[tail]),
             "m_scale": host(p.m_scale[first // 256:]), "v_scale": host(p.v_scale[first // 256:])}
        s["m"], s["v"] = O.decode_m(s["m_codes"], s["m_scale"]), O.decode_v(s["v_codes"], s["v_scale"])
        return s

    for t in (1, 2):
        before = view()
        plan.step()
        check_step(before, view(), cfg, p, t, first, 1.0, f"step {t}")
    assert float(w[5]) < 0 and torch.count_nonzero(w[: first - 512]).item() == 1
    norm = host(D.grad_norm([g]))[0]
    want = np.sqrt(np.sum(host(g[-700:]) ** 2) + 0.25 ** 2)
    assert abs(norm - want) <= 1.01 * U * want
