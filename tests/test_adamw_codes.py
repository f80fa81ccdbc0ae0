"""8-bit codes after a step, and large batches in the forms that other tests
reach only with small ones."""

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from oracle import adamw_oracle as O
from test_adamw import FORMS, U, host, snapshot, tensors

pytestmark = pytest.mark.gpu


def neighbours(code, want, signed, ctx):
    """A code that is not the oracle's is the one next to it in size, of the same sign unless it is zero."""
    code, want = code.astype(np.int64), want.astype(np.int64)
    size = (lambda c: c & 0x7F) if signed else (lambda c: c)
    gap = np.abs(size(code) - size(want))
    assert (gap <= 1).all(), (ctx, np.flatnonzero(gap > 1)[:5], code[gap > 1][:5], want[gap > 1][:5])
    if signed:
        flipped = ((code ^ want) & 0x80 != 0) & (size(code) != 0) & (size(want) != 0)
        assert not flipped.any(), (ctx, np.flatnonzero(flipped)[:5])
    return int((gap > 0).sum())


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("w,g,master", FORMS)
def test_codes_next_to_a_border_are_off_by_one_code(w, g, master, rounding):
    print(f"[case] neighbouring codes {w}/{g} master={master} {rounding}", flush=True)
    sizes = [1, 255, 300_001, 257, 4096 * 5]
    ps = tensors(sizes, w, g, "block8", master, seed=13)
    cfg = D.adamw_config_for(ps, rounding=rounding, seed=0x1234567890ABCDEF)
    plan = D.AdamWPlan(ps, cfg)
    firsts, off = plan.state_offsets(), 0
    for t in range(1, 4):
        before = [snapshot(p) for p in ps]
        plan.step()
        for i, p in enumerate(ps):
            b, a, n = before[i], snapshot(p), sizes[i]
            m, v = O.moments(b["m"], b["v"], b["g"], cfg.beta1, cfg.beta2)
            um = uv = 0.5
            if rounding == "stochastic":
                um, uv = [(r.astype(np.float64) * 16 + 8) / 2 ** 20
                          for r in O.random_bits(firsts[i] + np.arange(n), cfg.seed, t)]
            off += neighbours(a["m_codes"], O.encode_m(m, a["m_scale"], um), True, f"tensor {i} step {t} m")
            off += neighbours(a["v_codes"], O.encode_v(v, a["v_scale"], uv), False, f"tensor {i} step {t} v")
            p.g.copy_(-0.7 * p.g.roll(1))
    # Borders that a float32 error reaches: an error of 2^-20 of a code step on either side for most elements, 0.05 of
    # one for the few m in the subnormal range.
    assert off <= 0.01 * 3 * 2 * sum(sizes)


SIZES = [4096 * 300, 1_000_003, 4096 * 64 + 256, 2048 * 33]   # whole units, and ends inside a unit, group and block


def values(plan, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = plan.state_elems
    spread = torch.exp(2 * torch.randn(n, generator=gen, device="cuda"))
    return (torch.randn(n, generator=gen, device="cuda") * spread).to(dtype), spread.square().to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_32_bit_moments_take_and_give_large_values(dtype):
    """Exact both ways (bf16 values round once when given back)."""
    print(f"[case] 32-bit moments from {dtype}", flush=True)
    ps = tensors(SIZES, "bf16", "bf16", "f32", False, seed=14)
    plan = D.AdamWPlan(ps, D.adamw_config_for(ps))
    m, v = values(plan, dtype, 1)
    plan.set_state(m, v)
    for o, p in zip(plan.state_offsets(), ps):
        n = p.w.numel()
        assert torch.equal(p.m, m[o:o + n].float()) and torch.equal(p.v, v[o:o + n].float())
    for kind in (torch.float32, torch.bfloat16):
        a, b = plan.get_state(dtype=kind)
        for o, p in zip(plan.state_offsets(), ps):
            n = p.w.numel()
            assert torch.equal(a[o:o + n], m[o:o + n].to(kind)) and torch.equal(b[o:o + n], v[o:o + n].to(kind))
            end = o + -(-n // D.ADAMW_BLOCK) * D.ADAMW_BLOCK
            assert not a[o + n:end].any() and not b[o + n:end].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_8_bit_moments_take_large_values(dtype):
    """Nearest rounding over whole units: scales exact, codes the oracle's or next to them at a border."""
    print(f"[case] 8-bit moments from {dtype}", flush=True)
    ps = tensors(SIZES, "bf16", "bf16", "block8", False, seed=15)
    plan = D.AdamWPlan(ps, D.adamw_config_for(ps, rounding="nearest"))
    m, v = values(plan, dtype, 2)
    plan.set_state(m, v)
    off = 0
    for i, (o, p) in enumerate(zip(plan.state_offsets(), ps)):
        n = p.w.numel()
        mi, vi = host(m[o:o + n]), host(v[o:o + n])
        ms, vs = O.scales(mi, vi)
        np.testing.assert_array_equal(host(p.m_scale), ms)
        np.testing.assert_array_equal(host(p.v_scale), vs)
        off += neighbours(host(p.m), O.encode_m(mi, ms, 0.5), True, f"tensor {i} m")
        off += neighbours(host(p.v), O.encode_v(vi, vs, 0.5), False, f"tensor {i} v")
    assert off <= 2e-5 * 2 * sum(SIZES)   # quotients are within 2^-20 of a code step: twice that of them meet a border


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_gradients_beyond_the_cache(dtype):
    """More than 256 MB: every element counts once (random values; the plain
    sum of every tensor in binary64), whole and short leaves, both types."""
    print(f"[case] norm past the cache {dtype}", flush=True)
    per = 4 if dtype == torch.float32 else 2
    sizes = [(200 << 20) // per, (70 << 20) // per + 12345, 32768 // per, 32768 // per + 1, 7, 0, 3_000_001]
    gen = torch.Generator(device="cuda").manual_seed(16)
    grads = [torch.randn(n, generator=gen, device="cuda").to(dtype) for n in sizes]
    assert sum(g.numel() * per for g in grads) > 256 << 20
    each = [float(g.double().square().sum()) for g in grads]
    norms = torch.full((len(grads),), -1.0, device="cuda")
    plan = D.GradNormPlan(grads, 1.0, tensor_norms=norms)
    for _ in range(2):
        out = host(plan.run())
        want = np.sqrt(np.sum(each))
        assert abs(out[0] - want) <= 1.01 * U * want and abs(out[1] - 1 / want) <= 1.01 * U / want
        assert (np.abs(host(norms) - np.sqrt(each)) <= 1.01 * U * np.sqrt(each)).all()
