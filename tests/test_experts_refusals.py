"""Every refusal of the experts' calls by its message: what is wrong is named,
and not something else about the same call (CPU tensors are refused anyway).
On the GPU each call differs in one argument from one that is taken, with the
current stream (marshalled natively) and a given one (in Python)."""

import os

import pytest
import torch

import dimuon_newton_schulz_amd as D
from test_experts import PYTHON_REFUSALS, announce, rows_of

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")
HOST = "the tensors are on the CPU"

MESSAGES = {
    "ids_float": "ids is torch.float32", "ids_1d": r"ids must be \(tokens, top\)", "ids_strided": "ids must be contiguous",
    "ids_host": HOST, "experts": "experts 0 < 1", "routes_type": "routes must be ExpertRoutes", "routes_shapes": "routes.order has shape",
    "gather_host": HOST, "combine_host": HOST, "grad_host": HOST, "x_columns": "x has 8 columns, the weight 9",
    "x_dtype": "x is torch.float16", "w_dtype": "w is torch.bfloat16", "x_strided": "x: a row's elements must be consecutive",
    "x_expanded": "x: rows overlap", "x_1d": "x must have rows and columns", "bias_shape": "bias has shape",
    "residual_shape": "residual has shape", "no_offsets": "2 groups need offsets", "offsets_long": "offsets is torch.int64",
    "offsets_count": "offsets has shape", "activation": "activation must be one of", "out_shape": "out has shape",
    "linear_host": HOST, "nothing": "give at least one", "dx_without_w": "dx needs w", "dw_without_x": "dw needs x",
    "pre_missing": "through relu needs pre", "x_pre_missing": "through relu needs x_pre", "db_dtype": "db is torch.bfloat16",
    "dw_shape": "dw has shape", "dy_columns": "the weight has 6 rows, dy 7 columns", "workspace": "workspace must be uint8",
    "grad_workspace_host": HOST,
}


@built
@pytest.mark.parametrize("kind", sorted(PYTHON_REFUSALS))
def test_refusals_name_what_is_wrong(kind):
    with pytest.raises((ValueError, D.MuonError), match=MESSAGES[kind]):
        PYTHON_REFUSALS[kind]()


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def linear_grad_arguments():
    """Taken as they are: 12 rows, 16 to 24 columns, two groups."""
    return dict(dy=rows_of(12, 24, torch.bfloat16, 1), x=rows_of(12, 16, torch.bfloat16, 2), w=t(2, 24, 16), activation="silu",
                pre=t(12, 24), offsets=torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda"), dx=t(12, 16),
                dw=t(2, 24, 16, dtype=torch.float32), db=t(2, 24, dtype=torch.float32), x_activation="relu", x_pre=t(12, 16))


GRAD = {
    "dy_dtype": (lambda a: dict(dy=a["dy"].half()), "dy is torch.float16"),
    "dy_columns": (lambda a: dict(dy=t(12, 25)), "the weight has 24 rows, dy 25 columns"),
    "dy_strided": (lambda a: dict(dy=t(12, 48)[:, ::2]), "dy: a row's elements"),
    "dy_host": (lambda a: dict(dy=a["dy"].cpu()), "on cuda:0, the call's tensors on the CPU"),
    "pre": (lambda a: dict(pre=None), "through silu needs pre"),
    "pre_rows": (lambda a: dict(pre=t(11, 24)), "pre has shape"),
    "pre_dtype": (lambda a: dict(pre=a["pre"].float()), "pre is torch.float32"),
    "pre_strided": (lambda a: dict(pre=t(12, 48)[:, ::2]), "pre: a row's elements"),
    "x_pre": (lambda a: dict(x_pre=None), "through relu needs x_pre"),
    "x_pre_shape": (lambda a: dict(x_pre=t(12, 24)), "x_pre has shape"),
    "x_missing": (lambda a: dict(x=None), "dw needs x"),
    "x_columns": (lambda a: dict(x=t(12, 15)), "x has shape"),
    "x_dtype": (lambda a: dict(x=a["x"].float()), "x is torch.float32"),
    "x_host": (lambda a: dict(x=a["x"].cpu()), "x is on cpu"),
    "w_missing": (lambda a: dict(w=None), "dx needs w"),
    "w_dtype": (lambda a: dict(w=a["w"].float()), "w is torch.float32"),
    "w_strided": (lambda a: dict(w=t(2, 24, 32)[:, :, ::2]), "w: a row's elements"),
    "w_expanded": (lambda a: dict(w=t(1, 24, 16).expand(2, 24, 16)), "group stride 0 below a group's size"),
    "w_host": (lambda a: dict(w=a["w"].cpu()), "w is on cpu"),
    "dx_shape": (lambda a: dict(dx=t(12, 24)), "dx has shape"),
    "dx_dtype": (lambda a: dict(dx=a["dx"].float()), "dx is torch.float32"),
    "dw_shape": (lambda a: dict(dw=t(2, 16, 24)), "dw has shape"),
    "dw_dtype": (lambda a: dict(dw=a["dw"].half()), "dw is torch.float16"),
    "db_dtype": (lambda a: dict(db=a["db"].bfloat16()), "db is torch.bfloat16"),
    "db_shape": (lambda a: dict(db=t(24, 2, dtype=torch.float32)), "db has shape"),
    "db_strided": (lambda a: dict(db=t(2, 48, dtype=torch.float32)[:, ::2]), "db must be contiguous"),
    "offsets": (lambda a: dict(offsets=None), "2 groups need offsets"),
    "offsets_long": (lambda a: dict(offsets=a["offsets"].long()), "offsets is torch.int64"),
    "offsets_count": (lambda a: dict(offsets=a["offsets"][:2]), "offsets has shape"),
    "offsets_host": (lambda a: dict(offsets=a["offsets"].cpu()), "offsets is on cpu"),
    "activation": (lambda a: dict(activation="swish"), "activation must be one of"),
    "x_activation": (lambda a: dict(x_activation=4), "activation must be one of"),
    "nothing": (lambda a: dict(dx=None, dw=None, db=None), "give at least one"),
    "workspace_dtype": (lambda a: dict(workspace=t(1 << 16)), "workspace must be uint8"),
    "workspace_small": (lambda a: dict(workspace=t(256, dtype=torch.uint8)), "256 < [0-9]+ needed|256 bytes < [0-9]+ needed"),
    "workspace_shifted": (lambda a: dict(workspace=t(1 << 16, dtype=torch.uint8)[64:]), "not 256-byte aligned"),
    "workspace_strided": (lambda a: dict(workspace=t(1 << 16, dtype=torch.uint8)[::2]), "workspace must be a contiguous"),
    "workspace_host": (lambda a: dict(workspace=torch.zeros(1 << 16, dtype=torch.uint8)), "workspace is on cpu"),
    "dx_is_x": (lambda a: dict(dx=a["x"]), "overlaps"),
    "dx_is_dy": (lambda a: dict(dx=a["dy"][:, :16]), "overlaps"),
    "dw_is_w": (lambda a: dict(dw=a["w"], db=None), "overlaps"),
    "db_in_dw": (lambda a: dict(db=a["dw"].view(-1)[:48].view(2, 24)), "overlaps"),
}


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kind", sorted(GRAD))
def test_linear_grad_refusals_on_the_gpu(kind, given):
    announce(f"linear_grad refuses {kind}, {'given' if given else 'current'} stream")
    change, message = GRAD[kind]
    stream = torch.cuda.current_stream() if given else None
    a = linear_grad_arguments()
    D.linear_grad(**a, stream=stream)
    written = {k: a[k].clone() for k in ("dx", "dw", "db")}
    b = {**a, **change(a)}
    with pytest.raises((ValueError, D.MuonError), match=message):
        D.linear_grad(**b, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], v) for k, v in written.items())


def other_arguments():
    ids = torch.tensor([[0, 1], [1, 0], [1, 1]], dtype=torch.int32, device="cuda")
    r = D.expert_sort(ids, 2)
    return dict(ids=ids, r=r, x=rows_of(3, 16, torch.bfloat16, 1), xs=rows_of(6, 16, torch.bfloat16, 2), out=t(3, 16), outs=t(6, 16),
                weights=t(3, 2, dtype=torch.float32), dweights=t(3, 2, dtype=torch.float32))


def replaced(r, **kw):
    return D.ExpertRoutes(**{**dict(offsets=r.offsets, order=r.order, place=r.place), **kw})


OTHERS = {
    "sort_float": (lambda a, s: D.expert_sort(a["ids"].float(), 2, stream=s), "ids is torch.float32"),
    "sort_experts": (lambda a, s: D.expert_sort(a["ids"], 1025, stream=s), "experts 1025 above 1024"),
    "sort_strided": (lambda a, s: D.expert_sort(t(3, 4, dtype=torch.int32)[:, ::2], 2, stream=s), "ids must be contiguous"),
    "sort_routes": (lambda a, s: D.expert_sort(a["ids"], 3, routes=a["r"], stream=s), "routes are of 2 experts"),
    "sort_into_ids": (lambda a, s: D.expert_sort(a["ids"], 2, routes=replaced(a["r"], place=a["ids"]), stream=s), "overlaps"),
    "gather_rows": (lambda a, s: D.expert_gather(a["x"][:2], a["r"], stream=s), "x has shape"),
    "gather_out": (lambda a, s: D.expert_gather(a["x"], a["r"], out=t(5, 16), stream=s), "out has shape"),
    "gather_dtype": (lambda a, s: D.expert_gather(a["x"], a["r"], out=t(6, 16, dtype=torch.float32), stream=s), "out is torch.float32"),
    "gather_width": (lambda a, s: D.expert_gather(a["x"][:, :0], a["r"], stream=s), "width 0 < 1"),
    "gather_place": (lambda a, s: D.expert_gather(a["x"], replaced(a["r"], place=a["r"].place.long()), stream=s), "routes.place is"),
    "gather_offsets": (lambda a, s: D.expert_gather(a["x"], replaced(a["r"], offsets=a["r"].offsets[:1]), stream=s), "experts \\+ 1"),
    "gather_in_place": (lambda a, s: D.expert_gather(a["xs"][:3], a["r"], out=a["xs"], stream=s), "overlaps"),
    "combine_weights": (lambda a, s: D.expert_combine(a["xs"], a["r"], weights=t(3, 3, dtype=torch.float32), stream=s), "weights has shape"),
    "combine_weights_half": (lambda a, s: D.expert_combine(a["xs"], a["r"], weights=a["weights"].half(), stream=s), "weights is torch.float16"),
    "combine_residual": (lambda a, s: D.expert_combine(a["xs"], a["r"], residual=a["xs"], stream=s), "residual has shape"),
    "combine_out": (lambda a, s: D.expert_combine(a["xs"], a["r"], out=t(6, 16), stream=s), "out has shape"),
    "combine_shifted": (lambda a, s: D.expert_combine(a["xs"], a["r"], residual=t(4, 16).view(-1)[:48].view(3, 16),
                                                      out=a["xs"][2:5], stream=s), "overlaps"),
    "grad_dy": (lambda a, s: D.expert_combine_grad(a["xs"], a["xs"], a["weights"], a["r"], stream=s), "dy has shape"),
    "grad_dweights": (lambda a, s: D.expert_combine_grad(a["x"], a["xs"], a["weights"], a["r"], dys=a["outs"],
                                                         dweights=a["dweights"].bfloat16(), stream=s), "dweights is torch.bfloat16"),
    "grad_in_place": (lambda a, s: D.expert_combine_grad(a["x"], a["xs"], a["weights"], a["r"], dys=a["xs"], stream=s), "overlaps"),
    "grad_into_weights": (lambda a, s: D.expert_combine_grad(a["x"], a["xs"], a["weights"], a["r"], dys=a["outs"],
                                                             dweights=a["weights"], stream=s), "overlaps"),
    "linear_pre_is_out": (lambda a, s: D.linear(a["x"], t(16, 16), pre=a["out"], out=a["out"], stream=s), "overlaps"),
    "linear_pre_is_residual": (lambda a, s: D.linear(a["x"], t(16, 16), pre=a["out"], residual=a["out"], stream=s), "overlaps"),
    "linear_out_is_x": (lambda a, s: D.linear(a["x"], t(16, 16), out=a["x"], stream=s), "overlaps"),
    "linear_bias_dtype": (lambda a, s: D.linear(a["x"], t(16, 16), bias=t(16, dtype=torch.float32), stream=s), "bias is torch.float32"),
    "linear_no_columns": (lambda a, s: D.linear(a["x"][:, :0], t(16, 0), stream=s), "below 1"),
}


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kind", sorted(OTHERS))
def test_refusals_on_the_gpu(kind, given):
    announce(f"refusal {kind}, {'given' if given else 'current'} stream")
    call, message = OTHERS[kind]
    a = other_arguments()
    kept = {k: v.clone() for k, v in a.items() if k != "r"}
    with pytest.raises((ValueError, D.MuonError), match=message):
        call(a, torch.cuda.current_stream() if given else None)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], v) for k, v in kept.items())
