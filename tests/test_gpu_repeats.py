"""Identical steps give identical bits, over more repeats than one pair, with
a report that says what differs and where (the refill of a stage's LDS buffer
once raced with late reads of it, and one pair of steps rarely showed it)."""

import pytest
import torch

import dimuon_newton_schulz_amd as D

pytestmark = pytest.mark.gpu

BATCHES = {
    "square": ([(4096, 4096)] * 8, 8),
    "experts": ([(2048, 1408), (1408, 2048)] * 16, 8),
    "hidden": ([(768, 2304), (768, 768), (2304, 768)] * 12, 12),
    "small_square": ([(1024, 1024)] * 8, 24),      # 512 tiles of 128 x 128
    "odd": ([(513, 1300), (1300, 513), (640, 256)] * 6, 24),
}


def differences(name, first, again):
    """One line per tensor that differs: how many elements, the first few places, the largest difference."""
    lines = []
    for i, (a, b) in enumerate(zip(first, again)):
        for what in ("w", "mom"):
            x, y = getattr(a, what), getattr(b, what)
            off = (x.view(torch.int16) != y.view(torch.int16)).nonzero()
            if len(off):
                gap = (x.float() - y.float()).abs().max().item()
                lines.append(f"{name}: matrix {i} {tuple(x.shape)} {what}: {len(off)} elements differ, "
                             f"first at {off[:4].tolist()}, by at most {gap:.3g}")
    return lines


@pytest.mark.parametrize("variant", ["muon", "dimuon"])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_steps_repeat_bit_for_bit(name, variant):
    shapes, repeats = BATCHES[name]
    print(f"[case] {name} {variant}, {repeats} repeats", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(17)
    base = [tuple((torch.randn(s, generator=gen, device="cuda") * 0.02).bfloat16() for _ in range(3)) for s in shapes]
    first = None
    for k in range(repeats):
        params = [D.Param(w=w.clone(), g=g.clone(), mom=m.clone()) for w, g, m in base]
        plan = D.Plan(params, D.StepConfig(lr=0.02, momentum=0.95), dimuon=variant == "dimuon")
        plan.step()
        torch.cuda.synchronize()
        plan.close()
        if first is None:
            first = params
            continue
        lines = differences(name, first, params)
        assert not lines, f"repeat {k}:\n" + "\n".join(lines)
