"""A plan reads the addresses it was created with, so it has to keep that
memory whatever the caller does to its config, parameter and gradient objects
afterwards."""

import gc
import os

import pytest
import torch

import dimuon_newton_schulz_amd as D

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


@built
def test_copies_do_not_follow_the_callers_objects():
    w, g, m = (torch.ones(64, 64) for _ in range(3))
    p, cfg = D.Param(w, g, m, update_scale=2.0), D.StepConfig(lr=0.5)
    cfg.grad_scale = torch.ones(1)
    a = D.adamw_param(torch.ones(300), torch.ones(300), state="block8")
    copies = [D._own(x) for x in (p, cfg, a)]
    where = [c.data_ptr() for c in (copies[0].g, copies[1].grad_scale, copies[2].m_scale)]
    p.g, p.update_scale, cfg.grad_scale, cfg.lr, a.m_scale = torch.zeros(64, 64), 3.0, None, 0.1, None
    w.data = torch.zeros(8, 8)
    assert copies[0].update_scale == 2.0 and copies[1].lr == 0.5 and copies[2].m.dtype == torch.float8_e4m3fn
    assert [c.data_ptr() for c in (copies[0].g, copies[1].grad_scale, copies[2].m_scale)] == where
    assert copies[0].w.shape == (64, 64) and (copies[0].w == 1).all()
    assert isinstance(copies[0], D.Param) and isinstance(copies[1], D.StepConfig) and isinstance(copies[2], D.AdamWParam)


def take_memory(shapes):
    """Fills what the allocator may have got back with values that would show."""
    gc.collect()
    torch.cuda.synchronize()
    return [torch.full(s, 1e4, device="cuda", dtype=dt) for s in shapes for dt in (torch.float32, torch.bfloat16)]


@gpu
@pytest.mark.parametrize("kind", ["adamw", "muon", "dimuon"])
def test_a_plan_keeps_what_it_reads(kind):
    """Gradients, weights and the scale taken out of the caller's objects after the plan's creation."""
    print(f"[case] plan ownership {kind}", flush=True)
    results = []
    for dropped in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(6)
        scale = torch.tensor([0.25], device="cuda")
        shapes = [(40, 300), (8, 520)]
        if kind == "adamw":
            ps = [D.adamw_param(*(torch.randn(s, generator=gen, device="cuda") for _ in range(2))) for s in shapes]
            cfg = D.adamw_config_for(ps, grad_scale=scale)
            plan = D.AdamWPlan(ps, cfg)
        else:
            ps = [D.Param(*(torch.randn(s, generator=gen, device="cuda") for _ in range(3))) for s in shapes]
            cfg = D.config_for(ps, grad_scale=scale)
            plan = D.Plan(ps, cfg, dimuon=kind == "dimuon")
        weights = [p.w for p in ps]
        if dropped:
            cfg.grad_scale = None
            for p in ps:
                p.g = p.w = None
            del scale
            taken = take_memory([(1,), (2,), *shapes])
        plan.step()
        plan.step()
        torch.cuda.synchronize()
        results.append([w.clone() for w in weights])
        if dropped:
            del taken
    for x, y in zip(*results):
        assert torch.equal(x, y)


@gpu
def test_a_norm_plan_keeps_what_it_reads():
    print("[case] norm plan ownership", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(6)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in (70000, 513)]
    norms = torch.zeros(2, device="cuda")
    plan = D.GradNormPlan(grads, tensor_norms=norms)
    want = plan.run().clone(), norms.clone()
    plan.tensor_norms = None
    out = plan.out
    for g in grads:
        g.data = torch.empty(0, device="cuda")
    del grads, g
    taken = take_memory([(70000,), (513,), (2,)])
    plan.run()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(norms, want[1]) and taken
