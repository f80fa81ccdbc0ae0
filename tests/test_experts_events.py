"""Launch events of calls that have nothing to launch."""

import pytest
import torch

import dimuon_newton_schulz_amd as D
from test_experts import announce, rows_of

gpu = pytest.mark.gpu


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
