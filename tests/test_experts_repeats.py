"""A token that chooses one expert several times: every choice is a row of its own."""

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from oracle import expert_oracle as O
from test_experts import U, announce, f64, rows_of, within

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("tokens,top,experts", [(1, 4, 1), (70, 5, 2), (3000, 4, 3), (600, 20, 7)])
def test_one_expert_chosen_again(tokens, top, experts):
    announce(f"repeated choices {tokens} x {top} of {experts}")
    ids = torch.randint(-1, experts, (tokens, top), generator=torch.Generator().manual_seed(tokens))
    r = D.expert_sort(ids.cuda(), experts)
    offsets, order, place = O.sort(ids.numpy(), experts)
    for got, want in ((r.offsets, offsets), (r.order, order), (r.place, place)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    x, w = rows_of(tokens, 40, torch.float32, 1), rows_of(tokens, top, torch.float32, 2)
    xs = D.expert_gather(x, r, out=torch.zeros(tokens * top, 40, device="cuda"))
    np.testing.assert_array_equal(f64(xs), O.gather(f64(x), place, np.zeros((tokens * top, 40))))
    size = O.combine(np.abs(f64(xs)), place, np.abs(f64(w)), np.abs(f64(x)))
    within(D.expert_combine(xs, r, w, x), O.combine(f64(xs), place, f64(w), f64(x)), (top + 4) * U * size, "y")
    dys, dw = D.expert_combine_grad(x, xs, w, r, dys=torch.zeros_like(xs))
    want, want_w = O.combine_grad(f64(x), f64(xs), f64(w), place, np.zeros(xs.shape))
    _, size = O.combine_grad(np.abs(f64(x)), np.abs(f64(xs)), f64(w), place, np.zeros(xs.shape))
    within(dys, want, U * np.abs(want), "dys")
    within(dw, want_w, 44 * U * size, "dweights")
