"""muon_config_t's grad_scale stands where older callers had reserved words,
which nothing told them to clear: it counts only in a config that says so."""

import ctypes

import pytest
import torch

import dimuon_newton_schulz_amd as D

STRAY = 0x7F03A5C91D37   # what a caller's stack may hold: misaligned, no device address


def batch():
    arr = (D.MuonMatrix * 1)()
    arr[0].w, arr[0].g, arr[0].mom, arr[0].m, arr[0].n = 0x100000000, 0x110000000, 0x120000000, 64, 256
    arr[0].update_scale = 1.0
    return arr


def calls(lib, arr, cfg):
    handle = ctypes.c_void_p(0)
    for step in (lib.muon_step, lib.dimuon_step):
        yield step(arr, 1, ctypes.byref(cfg), None, 0, None)
    yield lib.muon_plan_create(arr, 1, ctypes.byref(cfg), 0, None, 0, None, ctypes.byref(handle))


@pytest.mark.parametrize("words", [(0, 0), (-1, -1), (1, 1), (0x5A5A5A5A, 0x5A5A5A5A)])
def test_words_that_a_caller_never_set_are_not_read(words):
    """A config filled by hand, field by field: what its last words hold is not looked at."""
    lib, arr = D.load_library(), batch()
    cfg = D.MuonConfig()
    cfg.lr, cfg.momentum, cfg.ns_steps, cfg.a, cfg.b, cfg.c = 0.02, 0.95, 5, 3.4445, -4.775, 2.0315
    cfg.w_dtype = cfg.g_dtype = cfg.mom_dtype = cfg.ns_dtype = D.MUON_BF16
    cfg.fields, cfg.reserved[0] = words
    cfg.grad_scale = STRAY
    out = ctypes.c_size_t(0)
    assert lib.muon_workspace_bytes(arr, 1, ctypes.byref(cfg), ctypes.byref(out)) == 0 and out.value
    for status in calls(lib, arr, cfg):   # all is well up to the missing workspace
        assert status == 3, lib.muon_last_error()


def test_default_configs_name_the_field():
    lib, arr = D.load_library(), batch()
    by_default = D.MuonConfig()
    lib.muon_config_default(ctypes.byref(by_default))
    from_python, _ = D.StepConfig().to_c()
    for cfg in (by_default, from_python):
        assert cfg.fields == D.MUON_CONFIG_FIELDS and not cfg.grad_scale
        for status in calls(lib, arr, cfg):
            assert status == 3
        cfg.grad_scale = STRAY
        for status in calls(lib, arr, cfg):
            assert status == 1 and b"grad_scale" in lib.muon_last_error()
    assert ctypes.sizeof(D.MuonConfig) == 80 and D.MuonConfig.fields.offset == 60   # as before grad_scale


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(8, 1000), (200, 300)])
def test_a_step_ignores_a_scale_that_the_config_does_not_name(shape):
    print(f"[case] unnamed grad_scale {shape}", flush=True)
    scale, got = torch.tensor([0.37], device="cuda"), {}
    for how in ("none", "unnamed", "named"):
        gen = torch.Generator(device="cuda").manual_seed(3)
        p = D.Param(*(torch.randn(shape, generator=gen, device="cuda").bfloat16() for _ in range(3)))
        cfg, _ = D.StepConfig(grad_scale=None if how == "none" else scale).to_c()
        if how == "unnamed":
            cfg.fields = 0
        arr, ws = D._marshal([p]), D.workspace_for([p], D.StepConfig())
        assert D.load_library().muon_step(arr, 1, ctypes.byref(cfg), ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream) == 0
        got[how] = (p.w, p.mom)
    assert all(torch.equal(a, b) for a, b in zip(got["none"], got["unnamed"]))
    assert not torch.equal(got["none"][1], got["named"][1])
