"""Views of one wide buffer's columns as a call's buffers: no byte is shared,
also where one of them has a single row (a batch of one token)."""

import pytest
import torch

import dimuon_newton_schulz_amd as D
from test_experts import announce, rows_of

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("tokens,top,width", [(1, 2, 8), (1, 1, 5), (2, 3, 16), (1, 6, 264)])
def test_columns_of_one_buffer(tokens, top, width, stream):
    announce(f"columns of one buffer: {tokens} x {top}, {width}, {'given' if stream else 'current'} stream")
    s = torch.cuda.current_stream() if stream else None   # (given: marshalled in Python)
    ids = torch.arange(tokens * top, device="cuda", dtype=torch.int32).view(tokens, top) % top
    r = D.expert_sort(ids, top)
    wide = rows_of(tokens * top, 3 * width, torch.bfloat16, 1)
    a, b, c = wide[:, :width], wide[:, width:2 * width], wide[:, 2 * width:]
    weights = rows_of(tokens, top, torch.float32, 2)
    for i, (x, xs) in enumerate(((a[:tokens], b), (b[:tokens], a), (c[:tokens], a))):
        keep = wide.clone()
        want = D.expert_gather(x.clone(), r)
        D.expert_gather(x, r, out=xs, stream=s)
        assert torch.equal(xs, want) and torch.equal(c, keep[:, 2 * width:]), i
    want = D.expert_combine(a.clone(), r, weights)
    D.expert_combine(a, r, weights, out=b[:tokens], stream=s)
    assert torch.equal(b[:tokens], want)
    dys, _ = D.expert_combine_grad(b[:tokens].clone(), a.clone(), weights, r)
    keep = wide.clone()
    D.expert_combine_grad(b[:tokens], a, weights, r, dys=c, stream=s)
    assert torch.equal(c, dys) and torch.equal(wide[:, :2 * width], keep[:, :2 * width])
    for y in (wide[:tokens, width - 1:2 * width - 1], wide[-tokens:, :width], wide[:tokens, :width]):
        with pytest.raises(D.MuonError, match="overlaps"):
            D.expert_combine(a, r, weights, out=y, stream=s)
    assert torch.equal(wide[:, :2 * width], keep[:, :2 * width])
