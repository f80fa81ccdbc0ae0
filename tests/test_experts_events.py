"""Calls of the experts' layers that have nothing to launch."""

import ctypes
import os

import pytest
import torch

import dimuon_newton_schulz_amd as D
from dimuon_newton_schulz_amd import experts as X
from test_experts import announce, rows_of

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


@gpu
def test_calls_without_rows_record_no_events():
    """The count is the last call's, not that of one before it."""
    announce("events of calls without rows")
    w = rows_of(8, 16, torch.float32, 1)
    none, x = torch.empty(0, 16, device="cuda"), rows_of(4, 16, torch.float32, 2)
    r = D.expert_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    weights = torch.empty(0, 2, device="cuda")
    with D.LaunchTimer(8) as t:
        for call in (lambda: D.linear(none, w), lambda: D.expert_gather(none, r), lambda: D.expert_combine(none, r),
                     lambda: D.expert_combine_grad(none, none, weights, r),
                     lambda: D.linear_grad(torch.empty(0, 8, device="cuda"), w=w, dx=none)):
            D.linear(x, w)
            assert t.recorded() == 2
            call()
            assert t.recorded() <= 1   # (the start, at most)


@built
def test_input_gradient_of_no_rows_is_nothing_to_do():
    """An empty dx has no address; with rows it is missing."""
    lib = D.load_library()
    a = X.LinearGradArgs(rows=0, in_=16, out=8, groups=1, w=1 << 32, w_stride=16, dx_stride=16, dtype=1, grad_dtype=1)
    assert lib.linear_grad(ctypes.byref(a), None, 0, None) == 0
    a.rows = 1
    assert lib.linear_grad(ctypes.byref(a), None, 0, None) == 1


@gpu
def test_input_gradient_of_no_rows():
    announce("dx of no rows")
    w, none, dy = rows_of(8, 16, torch.float32, 1), torch.empty(0, 16, device="cuda"), torch.empty(0, 8, device="cuda")
    assert D.linear_grad(dy, w=w, dx=none) == (none, None, None)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    D.linear_grad(dy, w=w.expand(2, 8, 16).contiguous(), activation="relu", pre=dy, offsets=off, dx=none)
