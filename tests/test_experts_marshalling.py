"""The experts' calls without the extension module that marshals them: the
rest of the package does not need it, and they go on in Python."""

import os
import subprocess
import sys

import pytest
import torch

import dimuon_newton_schulz_amd as D
from dimuon_newton_schulz_amd import experts as X
from test_experts import announce, rows_of, weight

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# What a program sees whose module cannot be imported (not built, or built for another torch).
WITHOUT = """
import sys, warnings
sys.modules["dimuon_newton_schulz_amd._binding"] = None
import torch
import dimuon_newton_schulz_amd as D
with warnings.catch_warnings():
    warnings.simplefilter("error")
    assert D.load_library().muon_abi_version() == 1
    p = D.Param(w=torch.zeros(8, 16), g=torch.zeros(8, 16), mom=torch.zeros(8, 16))
    assert D.muon_workspace_bytes([p], D.config_for([p])) > 0
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for _ in range(2):
        try:
            D.linear(torch.zeros(4, 8), torch.zeros(6, 9))
            raise SystemExit("not refused")
        except ValueError as e:
            assert "8 columns" in str(e), e
assert [w.category for w in seen] == [RuntimeWarning], seen
print("fine")
"""


@built
def test_package_without_the_extension_module():
    done = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip().endswith("fine"), done.stderr[-2000:]


@built
@pytest.mark.parametrize("field,value", [("torch_version", "1.2.3"), ("python_version", "2.7")])
def test_module_of_another_build_is_not_used(monkeypatch, field, value):
    from dimuon_newton_schulz_amd import _binding
    assert X._load_binding(D.load_library()) is _binding
    monkeypatch.setattr(_binding, field, value)
    with pytest.warns(RuntimeWarning, match="built for"):
        assert X._load_binding(D.load_library()) is not _binding


def test_library_is_linked_before_a_module_that_does_not_build(monkeypatch):
    from dimuon_newton_schulz_amd import build as B
    commands = []

    def no_module():
        raise RuntimeError("no host compiler")

    monkeypatch.setattr(B, "_run", lambda cmd: commands.append(cmd) or "")
    monkeypatch.setattr(B, "build_binding", no_module)
    monkeypatch.setattr(B.os, "replace", lambda a, b: None)
    with pytest.raises(RuntimeError, match="no host compiler"):
        B.build()
    assert commands[-1][-len(B.SOURCES):] == [os.path.join(B.BUILD, s.replace(".hip", ".o")) for s in B.SOURCES]


@gpu
def test_calls_without_the_extension_module(monkeypatch):
    """The same bits as with it."""
    def calls():
        r = D.expert_sort((torch.arange(90, device="cuda") * 7 % 5).view(30, 3), 5)
        x, w = rows_of(30, 64, torch.bfloat16, 1), weight(5, 48, 64, torch.bfloat16, 2)
        xs = D.expert_gather(x, r)
        pre = torch.zeros(90, 48, dtype=torch.bfloat16, device="cuda")
        ys = D.linear(xs, w, activation="silu", offsets=r.offsets, pre=pre)
        weights = rows_of(30, 3, torch.float32, 3)
        y = D.expert_combine(ys, r, weights)
        dys, dweights = D.expert_combine_grad(y, ys, weights, r)
        dx, dw = torch.zeros_like(xs), torch.zeros(5, 48, 64, device="cuda")
        D.linear_grad(dys, xs, w, activation="silu", pre=pre, offsets=r.offsets, dx=dx, dw=dw)
        return [r.offsets, r.order, r.place, xs, ys, y, dys, dweights, dx, dw]

    announce("without the extension module")
    want = calls()
    monkeypatch.setitem(sys.modules, "dimuon_newton_schulz_amd._binding", None)
    monkeypatch.delattr(D, "_binding")
    monkeypatch.setattr(X, "_fast", None)
    with pytest.warns(RuntimeWarning, match="_binding"):
        got = calls()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
