"""8-bit moments at the ends of the range that their scales allow.

v = u(code) * v_scale is rounded to float32.  Below 2^-126 that rounding is
absolute, by 2^-150 at most; the step between the smallest codes is
2^-34 * v_scale.  From v_scale = 2^-114 on, 2^-150 is at most a quarter of it,
so the nearest code is the one that the value came from.  For m the smallest
step is 2^-9 * m_scale, 2^-135 or more while m_scale is a normal number.
"""

import os

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from oracle import adamw_oracle as O
from test_adamw import check_step, host, snapshot

gpu = pytest.mark.gpu
F32_MAX = float(np.finfo(np.float32).max)


def v_scales():
    return [np.float32(np.ldexp(s, e)) for e in (-114, -113, -94, -20, 0, 1, 60, 127) for s in (1.0, 1.3, 2 - 2.0 ** -23)]


def m_scales():
    return [np.float32(np.ldexp(s, e)) for e in (-126, -125, -100, 0, 60, 119) for s in (1.0, 1.3, 2 - 2.0 ** -23)]


M_CODES = np.concatenate([np.arange(0, 0x79), np.arange(0x80, 0xF9)]).astype(np.uint8)   # |e4m3| up to 256
V_CODES = np.arange(0, 249, dtype=np.uint8)


def test_values_in_float32_have_the_code_they_came_from():
    for s in v_scales():
        v = O.decode_v(V_CODES, np.array([s], np.float64)).astype(np.float32)
        np.testing.assert_array_equal(O.encode_v(v, np.array([s], np.float64), 0.5), V_CODES, err_msg=str(s))
    for s in m_scales():
        m = O.decode_m(M_CODES, np.array([s], np.float64)).astype(np.float32)
        np.testing.assert_array_equal(O.encode_m(m, np.array([s], np.float64), 0.5), M_CODES, err_msg=str(s))
    # Below the bound they need not: the smallest values vanish.
    s = np.array([np.ldexp(1.3, -120)])
    v = O.decode_v(V_CODES, s).astype(np.float32)
    assert (O.encode_v(v, s, 0.5) != V_CODES).sum() > 10


def test_the_header_states_the_bound():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muon_mi355x.h")
    text = " ".join(open(path).read().replace("*", " ").split())
    assert "v's where v_scale is 2^-114 or more" in text and "codes of a block whose scales are normal float32" not in text


def filled(m_scale, v_scale, m_codes, v_codes):
    """One parameter whose block k holds all codes at scales k."""
    blocks = len(m_scale)
    m, v = np.zeros((blocks, 256), np.uint8), np.zeros((blocks, 256), np.uint8)
    m[:, :len(m_codes)], v[:, :len(v_codes)] = m_codes, v_codes
    p = D.adamw_param(torch.zeros(blocks * 256, device="cuda"), torch.zeros(blocks * 256, device="cuda"), state="block8")
    p.m.view(torch.uint8).copy_(torch.from_numpy(m.ravel()))
    p.v.copy_(torch.from_numpy(v.ravel()))
    p.m_scale.copy_(torch.from_numpy(np.asarray(m_scale, np.float32)))
    p.v_scale.copy_(torch.from_numpy(np.asarray(v_scale, np.float32)))
    return p


@gpu
@pytest.mark.parametrize("odd", [False, True])
def test_codes_survive_their_values_at_the_bounds(odd):
    """Every code at every scale of the lists, NaN codes among them (`odd`)."""
    print(f"[case] codes at the bounds, NaN codes {odd}", flush=True)
    vs, ms = v_scales(), m_scales()
    pairs = [(ms[i % len(ms)], vs[i % len(vs)]) for i in range(max(len(ms), len(vs)))]
    p = filled([a for a, _ in pairs], [b for _, b in pairs],
               np.append(M_CODES, [0x7F] if odd else []).astype(np.uint8), np.append(V_CODES, [255] if odd else []).astype(np.uint8))
    names = ("m", "v", "m_scale", "v_scale")
    before = {k: host(getattr(p, k)).copy() for k in names}
    plan = D.AdamWPlan([p], D.adamw_config_for([p]))
    m, v = plan.get_state()
    for got, want in ((m, O.decode_m(before["m"], before["m_scale"])), (v, O.decode_v(before["v"], before["v_scale"]))):
        np.testing.assert_array_equal(host(got), want.astype(np.float32).astype(np.float64))   # one rounding, to nearest
    plan.set_state(m, v)
    for k in names:
        np.testing.assert_array_equal(host(getattr(p, k)), before[k], err_msg=k)


@gpu
@pytest.mark.parametrize("beta2", [0.5, 0.999])
def test_small_v_keeps_its_denominator_above_eps(beta2):
    """v at its smallest code, v_scale at 2^-94: the root does not see zero."""
    print(f"[case] smallest denominators beta2={beta2}", flush=True)
    codes = np.concatenate([np.arange(1, 249), [248] * 8]).astype(np.uint8)
    m_codes = np.full(256, 0x28, np.uint8)
    m_codes[0] = 0x78   # 256, as in every block
    p = filled([2.0 ** -60] * 2, [2.0 ** -94, 1.7 * 2.0 ** -94], m_codes, codes)
    cfg = D.adamw_config_for([p], lr=1e-12, beta2=beta2, eps=1e-30, rounding="nearest")
    plan = D.AdamWPlan([p], cfg, step=4)
    before = snapshot(p)
    plan.step()
    after = snapshot(p)
    check_step(before, after, cfg, p, 5, 0, 1.0, "small v")
    # were any root zero, the step would be lr * m / eps, some 10^7 times this bound
    assert np.abs(after["w"]).max() < 1e-12 * np.abs(before["m"]).max() * 10 / np.sqrt(before["v"].min() * 0.5)
