"""A caller's workspace is checked before its address goes to the library:
kernels would read a host address, and the library takes the tensor's element
count as bytes."""

import os

import pytest
import torch

import dimuon_newton_schulz_amd as D

pytestmark = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")

GPU = torch.device("cuda", 0)


def test_workspaces_on_another_device_are_refused():
    host = torch.zeros(1 << 20, dtype=torch.uint8)
    for any_dtype in (False, True):
        with pytest.raises(ValueError, match="workspace"):
            D._check_workspace(host, GPU, any_dtype)
        D._check_workspace(host, host.device, any_dtype)
        D._check_workspace(None, GPU, any_dtype)


BAD = {
    "float32": lambda: torch.zeros(1 << 16),
    "int8": lambda: torch.zeros(1 << 20, dtype=torch.int8),
    "strided": lambda: torch.zeros(1 << 20, dtype=torch.uint8)[::2],
    "expanded": lambda: torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
    "a list": lambda: [0] * 1000,
}


def adamw_calls(ws):
    w = torch.zeros(300, dtype=torch.bfloat16)
    p = [D.adamw_param(w, w.clone())]
    cfg = D.adamw_config_for(p)
    return {"adamw_step": lambda: D.adamw_step(p, cfg, 1, workspace=ws),
            "AdamWPlan": lambda: D.AdamWPlan(p, cfg, workspace=ws),
            "grad_norm": lambda: D.grad_norm([w], workspace=ws),
            "GradNormPlan": lambda: D.GradNormPlan([w], workspace=ws)}


@pytest.mark.parametrize("kind", sorted(BAD))
@pytest.mark.parametrize("call", ["adamw_step", "AdamWPlan", "grad_norm", "GradNormPlan"])
def test_adamw_and_norm_refuse_a_workspace_that_is_not_bytes(call, kind):
    with pytest.raises(ValueError, match="workspace"):
        adamw_calls(BAD[kind]())[call]()


@pytest.mark.parametrize("kind", ["strided", "expanded", "a list"])
@pytest.mark.parametrize("call", ["muon_step", "dimuon_step", "Plan"])
def test_muon_refuses_a_workspace_that_is_not_contiguous(call, kind):
    p = [D.Param(*(torch.zeros(64, 256, dtype=torch.bfloat16) for _ in range(3)))]
    cfg = D.StepConfig()
    with pytest.raises(ValueError, match="workspace"):
        if call == "Plan":
            D.Plan(p, cfg, False, workspace=BAD[kind]())
        else:
            getattr(D, call)(p, cfg, workspace=BAD[kind]())
