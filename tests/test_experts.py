"""The experts' operators (sort, gather, combine and its gradient; products
over groups of rows and their gradients): the oracle against differences and
refusals on the CPU, results on the GPU against the float64 oracle.

Bounds count roundings.  U = 2^-24 is half a float32 step relative to the
value, H(dtype) half a step of the stored type (U, or 2^-8 for bf16).
  sums of K products in float32, in any order: (K + 4) U of the sum of their
      absolute values (products of two bf16 values are exact; + 4: the bias,
      the residual, and the operands of those sums)
  activations and slopes: expf and erfcf within a few ulps, the exponent
      z + 0.044715 z^3 within 6 U of itself, which moves sigmoid by at most
      u sigmoid (1 - sigmoid) 6 U < 2 U: 32 U (1 + |z|) for both, and 1.2
      times the error of z (no slope is above 1.13)
  dz is rounded to the dtype: H of it, and 64 U (1 + |z|) of dy from the slope
  every stored value: H of itself
"""

import ctypes
import os
import sys

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from dimuon_newton_schulz_amd import experts as X
from oracle import expert_oracle as O

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def announce(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    err = np.abs(f64(got) - want)
    if err.size == 0:
        return
    assert np.isfinite(err).all(), f"{what}: not finite at {np.argwhere(~np.isfinite(err))[:4].tolist()}"
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"{what}{list(map(int, worst))}: off by {err[worst]:.3e}, bound {bound[worst]:.3e}, " \
                                 f"{int((err > bound).sum())} of {err.size} outside"


# ---------------------------------------------------------------------------
# CPU: the oracle
# ---------------------------------------------------------------------------
def test_oracle_sort_is_stable_and_drops():
    ids = np.array([[2, 0], [0, 7], [2, -1], [0, 2]])
    offsets, order, place = O.sort(ids, 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert order.tolist() == [1, 2, 6, 0, 4, 7, -1, -1]
    assert place.tolist() == [[3, 0], [1, -1], [4, -1], [2, 5]]


@pytest.mark.parametrize("act", sorted(D.ACTIVATIONS))
def test_oracle_slopes_match_differences(act):
    z = np.linspace(-6, 6, 241) + 0.0125   # (no sample at 0, where relu has a corner)
    h = 1e-5
    want = (O.activation(act, z + h) - O.activation(act, z - h)) / (2 * h)
    # central differences: h^2 / 6 of the third derivative (below 2 for all), and 1e-16 |act| / h
    np.testing.assert_allclose(O.slope(act, z), want, atol=1e-9)


def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(1)
    rows, inn, out, offsets = 7, 5, 4, [1, 4, 4, 6]
    x, w = rng.standard_normal((rows, inn)), rng.standard_normal((3, out, inn))
    b, c = rng.standard_normal((3, out)), rng.standard_normal((rows, out))
    x_pre = rng.standard_normal((rows, inn))

    def loss(x_pre, w, b):
        y, _ = O.linear(O.activation("silu", x_pre), w, b, "gelu_tanh", None, offsets)
        return float((y * c).sum())

    x = O.activation("silu", x_pre)
    _, pre = O.linear(x, w, b, "gelu_tanh", None, offsets)
    dx, dw, db = O.linear_grad(c, x, w, "gelu_tanh", pre, offsets, "silu", x_pre)
    for value, grad, name in ((x_pre, dx, "x_pre"), (w, dw, "w"), (b, db, "b")):
        num = np.zeros_like(value)
        for i in np.ndindex(value.shape):
            kept = value[i]
            value[i] = kept + 1e-6
            up = loss(x_pre, w, b)
            value[i] = kept - 1e-6
            num[i] = (up - loss(x_pre, w, b)) / 2e-6
            value[i] = kept
        np.testing.assert_allclose(grad, num, atol=2e-8, err_msg=name)   # 1e-15 of a loss of about 10 over 2e-6


def test_oracle_combine_gradient_matches_differences():
    rng = np.random.default_rng(2)
    place = np.array([[0, 2], [-1, 1], [3, -1]])
    ys, w, c = rng.standard_normal((6, 3)), rng.standard_normal((3, 2)), rng.standard_normal((3, 3))
    dys, dw = O.combine_grad(c, ys, w, place, np.zeros((6, 3)))
    for value, grad in ((ys, dys), (w, dw)):
        for i in np.ndindex(value.shape):
            kept = value[i]
            value[i] = kept + 0.5   # linear in each: exact up to rounding
            up = (O.combine(ys, place, w) * c).sum()
            value[i] = kept - 0.5
            assert abs(up - (O.combine(ys, place, w) * c).sum() - grad[i]) < 1e-12
            value[i] = kept


# ---------------------------------------------------------------------------
# CPU: refusals (nothing is enqueued; the addresses are never used)
# ---------------------------------------------------------------------------
BASE, STEP = 0x100000000, 0x10000000


def fake_routes(tokens=100, top=2, experts=8):
    return X.ExpertRoutesC(BASE, BASE + STEP, BASE + 2 * STEP, tokens, top, experts)


SORT_REFUSALS = {"null_ids": 1, "null_routes": 1, "null_place": 1, "tokens": 1, "top": 1, "experts0": 1, "experts_many": 6, "top_many": 6,
                 "slots": 6, "id_bytes": 2, "alias": 4, "alias_ids": 4, "misaligned": 1, "ws_null": 3, "ws_small": 3,
                 "ws_misaligned": 3, "ws_alias": 4}


@built
@pytest.mark.parametrize("kind", sorted(SORT_REFUSALS))
def test_expert_sort_refusals(kind):
    lib, r, ids, id_bytes, ws, ws_bytes = D.load_library(), fake_routes(), BASE + 3 * STEP, 8, None, 0
    if kind.startswith("ws"):
        r.tokens, ws, ws_bytes = 100000, BASE + 5 * STEP, 1 << 30
    if kind == "null_ids":
        ids = None
    elif kind == "null_routes":
        r = None
    elif kind == "null_place":
        r.place = None
    elif kind == "tokens":
        r.tokens = -1
    elif kind == "top":
        r.top = 0
    elif kind == "experts0":
        r.experts = 0
    elif kind == "experts_many":
        r.experts = 1025
    elif kind == "top_many":
        r.top = 1025
    elif kind == "slots":
        r.tokens, r.top = 1 << 29, 3
    elif kind == "id_bytes":
        id_bytes = 2
    elif kind == "alias":
        r.order = r.place + 400
    elif kind == "alias_ids":
        ids = r.order + 32
    elif kind == "misaligned":
        r.offsets += 2
    elif kind == "ws_null":
        ws = None
    elif kind == "ws_small":
        ws_bytes = 256
    elif kind == "ws_misaligned":
        ws += 16
    elif kind == "ws_alias":
        ws = r.place + 256
    st = lib.expert_sort(ids, id_bytes, None if r is None else ctypes.byref(r), ws, ws_bytes, None)
    assert st == SORT_REFUSALS[kind], (st, lib.muon_last_error())
    assert lib.muon_last_error()


MOVE_REFUSALS = {"null": 1, "dtype": 2, "width0": 1, "width_many": 6, "stride": 1, "stride_many": 6, "misaligned": 1,
                 "alias": 4, "weights_dtype": 2, "alias_place": 4}


@built
@pytest.mark.parametrize("call", ["gather", "combine", "combine_grad"])
@pytest.mark.parametrize("kind", sorted(MOVE_REFUSALS))
def test_expert_rows_refusals(kind, call):
    if call == "gather" and kind == "weights_dtype":
        pytest.skip("no weights")
    lib, r = D.load_library(), fake_routes()
    a = [BASE + i * STEP for i in range(3, 9)]
    width, ld, dt, w_dt = 64, 64, 1, 0
    if kind == "null":
        a[0] = None
    elif kind == "dtype":
        dt = 5
    elif kind == "width0":
        width = 0
    elif kind == "width_many":
        width, ld = 65537, 65544
    elif kind == "stride":
        ld = 63
    elif kind == "stride_many":
        ld = (1 << 20) + 8
    elif kind == "misaligned":
        a[0] += 1
    elif kind == "alias":
        a[1] = a[0] + 64
        a[2] = a[0] + 128
        a[3] = a[0] + 192
    elif kind == "alias_place":
        a[1] = a[2] = a[3] = r.place + 16
    elif kind == "weights_dtype":
        w_dt = 9
    rp = ctypes.byref(r)
    if call == "gather":
        st = lib.expert_gather(a[0], ld, width, dt, rp, a[1], ld, None)
    elif call == "combine":
        st = lib.expert_combine(a[0], ld, width, dt, rp, a[4], w_dt, a[2], ld, a[1], ld, None)
    else:
        st = lib.expert_combine_grad(a[0], ld, a[4], ld, width, dt, rp, a[5], w_dt, a[1], ld, a[2], None)
    assert st == MOVE_REFUSALS[kind], (st, lib.muon_last_error())


def fake_linear(**kw):
    a = X.LinearArgs(rows=100, in_=64, out=32, groups=4, offsets=BASE, dtype=1, activation=0, x=BASE + STEP, x_stride=64,
                     w=BASE + 2 * STEP, w_stride=64, w_group_stride=2048, bias=BASE + 3 * STEP, residual=BASE + 4 * STEP,
                     residual_stride=32, y=BASE + 5 * STEP, y_stride=32, pre=BASE + 6 * STEP, pre_stride=32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


LINEAR_REFUSALS = {
    "rows": (dict(rows=-1), 1), "rows_many": (dict(rows=1 << 30), 6), "in0": (dict(in_=0), 1),
    "out_many": (dict(out=65537), 6), "groups0": (dict(groups=0), 1), "groups_many": (dict(groups=4097), 6),
    "no_offsets": (dict(offsets=None), 1), "dtype": (dict(dtype=3), 2), "activation": (dict(activation=5), 1),
    "null_x": (dict(x=None), 1), "null_w": (dict(w=None), 1), "null_y": (dict(y=None), 1),
    "stride": (dict(x_stride=63), 1), "group_stride": (dict(w_group_stride=2047), 1),
    "stride_many": (dict(y_stride=(1 << 20) + 1), 6), "misaligned": (dict(bias=BASE + 3 * STEP + 1), 1),
    "y_on_x": (dict(y=BASE + STEP + 64), 4), "pre_on_y": (dict(pre=BASE + 5 * STEP), 4),
    "y_on_shifted_residual": (dict(y=BASE + 4 * STEP + 64), 4), "y_on_w": (dict(y=BASE + 2 * STEP + 4096), 4),
    "too_large": (dict(rows=(1 << 30) - 1, out=65536, y_stride=65536, residual=None, pre=None, y=1 << 60), 6),
}


@built
@pytest.mark.parametrize("kind", sorted(LINEAR_REFUSALS))
def test_linear_refusals(kind):
    kw, want = LINEAR_REFUSALS[kind]
    lib, a = D.load_library(), fake_linear(**kw)
    if kind == "too_large":
        a.groups, a.offsets, a.bias, a.w_group_stride = 1, None, None, 65536 * 64
        a.x, a.w = 1 << 50, 1 << 40
    st = lib.linear_forward(ctypes.byref(a), None)
    assert st == want, (st, lib.muon_last_error())
    assert lib.linear_forward(None, None) == 1


def fake_grad(**kw):
    a = X.LinearGradArgs(rows=100, in_=64, out=32, groups=4, offsets=BASE, dtype=1, grad_dtype=0, activation=4,
                         x_activation=1, dy=BASE + STEP, dy_stride=32, pre=BASE + 2 * STEP, pre_stride=32,
                         x=BASE + 3 * STEP, x_stride=64, w=BASE + 4 * STEP, w_stride=64, w_group_stride=2048,
                         x_pre=BASE + 5 * STEP, x_pre_stride=64, dx=BASE + 6 * STEP, dx_stride=64,
                         dw=BASE + 7 * STEP, dw_stride=64, dw_group_stride=2048, db=BASE + 8 * STEP)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


GRAD_REFUSALS = {
    "nothing": (dict(dx=None, dw=None, db=None), 1), "null_dy": (dict(dy=None), 1), "null_pre": (dict(pre=None), 1),
    "null_x": (dict(x=None), 1), "null_w": (dict(w=None), 1), "null_x_pre": (dict(x_pre=None), 1),
    "grad_dtype": (dict(grad_dtype=4), 2), "x_activation": (dict(x_activation=-1), 1),
    "dw_stride": (dict(dw_stride=60), 1), "dw_groups": (dict(dw_group_stride=1024), 1),
    "dx_on_dy": (dict(dx=BASE + STEP), 4), "dw_on_w": (dict(dw=BASE + 4 * STEP), 4), "db_in_dw": (dict(db=BASE + 7 * STEP), 4),
    "dx_on_x": (dict(dx=BASE + 3 * STEP), 4),
    "db_many": (dict(out=65536, groups=4096, dy_stride=65536, pre_stride=65536, dx=None, dw=None, rows=10), 6), "ws_null": ({}, 3), "ws_small": ({}, 3), "ws_misaligned": ({}, 3),
    "ws_alias": ({}, 4),
}


@built
@pytest.mark.parametrize("kind", sorted(GRAD_REFUSALS))
def test_linear_grad_refusals(kind):
    kw, want = GRAD_REFUSALS[kind]
    lib, a, ws, ws_bytes = D.load_library(), fake_grad(**kw), 0x700000000000, 1 << 40
    if kind == "ws_null":
        ws = None
    elif kind == "ws_small":
        ws_bytes = 4096
    elif kind == "ws_misaligned":
        ws += 64
    elif kind == "ws_alias":
        ws = BASE + 7 * STEP + 256
    st = lib.linear_grad(ctypes.byref(a), ws, ws_bytes, None)
    assert st == want, (st, lib.muon_last_error())


@built
def test_columns_of_one_buffer_do_not_overlap():
    """Views of one wide buffer's columns pass the check (the call then fails on the NULL workspace)."""
    lib = D.load_library()
    a = fake_grad(dy_stride=160, dx=BASE + STEP + 64, dx_stride=160, x_activation=0)
    assert lib.linear_grad(ctypes.byref(a), None, 0, None) == 3
    a.dx = BASE + STEP + 48
    assert lib.linear_grad(ctypes.byref(a), 0x700000000000, 1 << 40, None) == 4


@built
def test_workspace_sizes():
    lib, n = D.load_library(), ctypes.c_size_t(7)
    assert lib.expert_sort_workspace_bytes(8192, 1, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.expert_sort_workspace_bytes(8193, 1, 64, ctypes.byref(n)) == 0 and n.value >= 9 * 65 * 4
    a = fake_grad(activation=0, db=None)
    assert lib.linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0
    a.activation = 1
    assert lib.linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value >= 100 * 32 * 2
    assert lib.linear_grad_workspace_bytes(ctypes.byref(a), None) == 1


T = torch.zeros
PYTHON_REFUSALS = {
    "ids_float": lambda: D.expert_sort(T(4, 2), 8),
    "ids_1d": lambda: D.expert_sort(T(4, dtype=torch.int32), 8),
    "ids_strided": lambda: D.expert_sort(T(4, 4, dtype=torch.int32)[:, ::2], 8),
    "ids_host": lambda: D.expert_sort(T(4, 2, dtype=torch.int32), 8),
    "experts": lambda: D.expert_sort(T(4, 2, dtype=torch.int32), 0),
    "routes_type": lambda: D.expert_gather(T(4, 8), None),
    "routes_shapes": lambda: D.expert_gather(T(4, 8), D.ExpertRoutes(T(9).int(), T(7).int(), T(4, 2).int())),
    "gather_host": lambda: D.expert_gather(T(4, 8), ROUTES()),
    "combine_host": lambda: D.expert_combine(T(8, 8), ROUTES()),
    "grad_host": lambda: D.expert_combine_grad(T(4, 8), T(8, 8), T(4, 2), ROUTES()),
    "x_columns": lambda: D.linear(T(4, 8), T(6, 9)),
    "x_dtype": lambda: D.linear(T(4, 8).half(), T(6, 8).half()),
    "w_dtype": lambda: D.linear(T(4, 8), T(6, 8).bfloat16()),
    "x_strided": lambda: D.linear(T(4, 16)[:, ::2], T(6, 8)),
    "x_expanded": lambda: D.linear(T(1, 8).expand(4, 8), T(6, 8)),
    "x_1d": lambda: D.linear(T(8), T(6, 8)),
    "bias_shape": lambda: D.linear(T(4, 8), T(6, 8), bias=T(8)),
    "residual_shape": lambda: D.linear(T(4, 8), T(6, 8), residual=T(4, 8)),
    "no_offsets": lambda: D.linear(T(4, 8), T(2, 6, 8)),
    "offsets_long": lambda: D.linear(T(4, 8), T(2, 6, 8), offsets=T(3).long()),
    "offsets_count": lambda: D.linear(T(4, 8), T(2, 6, 8), offsets=T(4).int()),
    "activation": lambda: D.linear(T(4, 8), T(6, 8), activation="swish"),
    "out_shape": lambda: D.linear(T(4, 8), T(6, 8), out=T(4, 8)),
    "linear_host": lambda: D.linear(T(4, 8), T(6, 8)),
    "nothing": lambda: D.linear_grad(T(4, 6)),
    "dx_without_w": lambda: D.linear_grad(T(4, 6), dx=T(4, 8), dw=T(6, 8), x=T(4, 8)),
    "dw_without_x": lambda: D.linear_grad(T(4, 6), dw=T(6, 8)),
    "pre_missing": lambda: D.linear_grad(T(4, 6), x=T(4, 8), dw=T(6, 8), activation="relu"),
    "x_pre_missing": lambda: D.linear_grad(T(4, 6), w=T(6, 8), dx=T(4, 8), x_activation="relu"),
    "db_dtype": lambda: D.linear_grad(T(4, 6), x=T(4, 8), dw=T(6, 8), db=T(6).bfloat16()),
    "dw_shape": lambda: D.linear_grad(T(4, 6), x=T(4, 8), w=T(6, 8), dw=T(8, 6)),
    "dy_columns": lambda: D.linear_grad(T(4, 7), x=T(4, 8), dw=T(6, 8)),
    "workspace": lambda: D.linear_grad(T(4, 6), x=T(4, 8), dw=T(6, 8), workspace=T(1 << 12)),
    "grad_workspace_host": lambda: D.linear_grad(T(4, 6), x=T(4, 8), dw=T(6, 8)),
}


def ROUTES():
    return D.ExpertRoutes(T(9).int(), T(8).int(), T(4, 2).int())


@built
@pytest.mark.parametrize("kind", sorted(PYTHON_REFUSALS))
def test_python_refusals(kind):
    with pytest.raises((ValueError, D.MuonError)):
        PYTHON_REFUSALS[kind]()


# ---------------------------------------------------------------------------
# GPU: sort and rows
# ---------------------------------------------------------------------------
def make_ids(tokens, top, experts, drop, seed, dtype):
    """Distinct experts per token; a part dropped through numbers on either side of the range."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((tokens, experts)) + 0.4 * np.sin(np.arange(experts)), axis=1)[:, :top].astype(np.int64)
    bad = np.array([-1, experts, -2 ** 31, 2 ** 31 - 1] + ([2 ** 40, -2 ** 40, 2 ** 32] if dtype == torch.int64 else []))
    ids = np.where(rng.random(ids.shape) < drop, rng.choice(bad, ids.shape), ids)
    return torch.from_numpy(ids.reshape(tokens, top)).to(dtype)


SORTS = [(1, 1, 1, 0.0, "i64"), (1, 1, 1, 1.0, "i32"), (0, 2, 5, 0.0, "i32"), (8, 6, 64, 0.0, "i64"), (63, 1, 3, 0.2, "i32"),
         (64, 1, 2, 0.0, "i64"), (65, 2, 7, 0.3, "i64"), (1000, 3, 37, 0.14, "i32"), (1024, 8, 128, 0.0, "i64"),
         (8193, 1, 1, 0.0, "i32"), (4097, 2, 64, 0.1, "i64"), (1500, 7, 1024, 0.05, "i64"), (40, 3, 1024, 0.5, "i32"),
         (300000, 1, 9, 0.5, "i32"), (9000, 1, 4, 1.0, "i64"),
         (1100000, 2, 5, 0.1, "i32"), (2730, 3, 200, 0.1, "i64"), (2731, 3, 1023, 0.3, "i32")]


@gpu
@pytest.mark.parametrize("tokens,top,experts,drop,kind", SORTS)
def test_expert_sort(tokens, top, experts, drop, kind):
    announce(f"sort {tokens} x {top} of {experts}, drop {drop}, {kind}")
    ids = make_ids(tokens, top, experts, drop, tokens + experts, {"i32": torch.int32, "i64": torch.int64}[kind])
    got = D.expert_sort(ids.cuda(), experts)
    offsets, order, place = O.sort(ids.numpy(), experts)
    np.testing.assert_array_equal(got.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(got.order.cpu().numpy(), order)
    np.testing.assert_array_equal(got.place.cpu().numpy(), place)


def routed(tokens, top, experts, drop, seed=5):
    ids = make_ids(tokens, top, experts, drop, seed, torch.int32)
    offsets, order, place = O.sort(ids.numpy(), experts)
    r = D.ExpertRoutes(*(torch.from_numpy(v.astype(np.int32)).cuda() for v in (offsets, order, place)))
    return r, offsets, place


def rows_of(n, width, dtype, seed, pad=0, std=1.0):
    """n rows on the GPU, `pad` more columns in memory than in the view."""
    gen = torch.Generator().manual_seed(seed)
    wide = (torch.randn(n, width + pad, generator=gen) * std).to(dtype).cuda()
    return wide[:, :width]


WIDTHS = [(1, 0), (8, 0), (16, 8), (129, 0), (96, 3), (769, 0), (2048, 0), (2056, 16)]


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width,pad", WIDTHS)
def test_expert_gather(width, pad, dtype):
    tokens, top, experts = 133, 3, 11
    announce(f"gather {tokens} x {width} (+{pad}) {dtype}")
    r, offsets, place = routed(tokens, top, experts, 0.2)
    x = rows_of(tokens, width, DT[dtype], 1, pad)
    out = rows_of(tokens * top, width, DT[dtype], 2, pad)
    before = f64(out)
    assert D.expert_gather(x, r, out=out) is out
    np.testing.assert_array_equal(f64(out), O.gather(f64(x), place, before))
    fresh = D.expert_gather(x, r)
    n = int(offsets[-1])
    assert torch.equal(fresh[:n], out[:n])


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width,pad", WIDTHS)
@pytest.mark.parametrize("how", ["plain", "weights_f32", "weights_bf16", "residual", "in_place"])
def test_expert_combine(width, pad, how, dtype):
    tokens, top, experts = 67, 5, 9
    announce(f"combine {tokens} x {width} (+{pad}) {dtype} {how}")
    r, _, place = routed(tokens, top, experts, 0.3)
    dt = DT[dtype]
    ys = rows_of(tokens * top, width, dt, 3, pad)
    w = None if how == "plain" else rows_of(tokens, top, DT["bf16" if how == "weights_bf16" else "f32"], 4)
    res = rows_of(tokens, width, dt, 5, pad) if how in ("residual", "in_place") else None
    want = O.combine(f64(ys), place, f64(w), f64(res))
    size = O.combine(np.abs(f64(ys)), place, None if w is None else np.abs(f64(w)), None if res is None else np.abs(f64(res)))
    got = D.expert_combine(ys, r, weights=w, residual=res, out=res if how == "in_place" else None)
    within(got, want, (top + 4) * U * size + half(dt) * np.abs(want), "y")


@gpu
@pytest.mark.parametrize("dtype,w_dtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("width,pad", WIDTHS)
def test_expert_combine_grad(width, pad, dtype, w_dtype):
    tokens, top, experts = 71, 4, 6
    announce(f"combine_grad {tokens} x {width} (+{pad}) {dtype}, weights {w_dtype}")
    r, _, place = routed(tokens, top, experts, 0.3)
    dt, wt = DT[dtype], DT[w_dtype]
    dy, ys, w = rows_of(tokens, width, dt, 6, pad), rows_of(tokens * top, width, dt, 7, pad), rows_of(tokens, top, wt, 8)
    dys = rows_of(tokens * top, width, dt, 9, pad)
    before = f64(dys)
    want, want_w = O.combine_grad(f64(dy), f64(ys), f64(w), place, before)
    _, size_w = O.combine_grad(np.abs(f64(dy)), np.abs(f64(ys)), f64(w), place, before)
    _, dw = D.expert_combine_grad(dy, ys, w, r, dys=dys)
    touched = np.zeros(len(before), bool)
    touched[place[place >= 0]] = True
    np.testing.assert_array_equal(f64(dys)[~touched], before[~touched])
    within(dys, want, (U + half(dt)) * np.abs(want), "dys")
    within(dw, want_w, (width + 4) * U * size_w + half(wt) * np.abs(want_w), "dweights")


@gpu
@pytest.mark.parametrize("tokens,top", [(1, 1), (1, 8), (5000, 2), (3, 16), (2500, 11)])
def test_expert_rows_sizes(tokens, top):
    """One token, many tokens, more choices than are handled at once, and
    choices that are all dropped."""
    for drop in (0.0, 1.0):
        announce(f"rows {tokens} x {top}, drop {drop}")
        r, _, place = routed(tokens, top, 16, drop)
        x, w = rows_of(tokens, 264, torch.bfloat16, 1), rows_of(tokens, top, torch.float32, 2)
        xs = D.expert_gather(x, r, out=torch.full((tokens * top, 264), 7.0, dtype=x.dtype, device="cuda"))
        np.testing.assert_array_equal(f64(xs), O.gather(f64(x), place, np.full((tokens * top, 264), 7.0)))
        want = O.combine(f64(xs), place, f64(w), f64(x))
        size = O.combine(np.abs(f64(xs)), place, np.abs(f64(w)), np.abs(f64(x)))
        within(D.expert_combine(xs, r, w, x), want, (top + 4) * U * size + 2.0 ** -8 * np.abs(want), "y")
        _, dw = D.expert_combine_grad(x, xs, w, r)
        _, want = O.combine_grad(f64(x), f64(xs), f64(w), place, np.zeros(xs.shape))
        _, size = O.combine_grad(np.abs(f64(x)), np.abs(f64(xs)), f64(w), place, np.zeros(xs.shape))
        within(dw, want, (268 + 1) * U * size, "dweights")


# ---------------------------------------------------------------------------
# GPU: products
# ---------------------------------------------------------------------------
def split(kind, rows, groups, seed):
    """Offsets of `groups` groups over `rows` rows; None: a plain layer."""
    if kind == "layer":
        return None
    rng = np.random.default_rng(seed)
    if kind == "empty":       # no group has a row
        return np.zeros(groups + 1, int)
    if kind == "one":         # all rows in one group in the middle
        o = np.zeros(groups + 1, int)
        o[groups // 2 + 1:] = rows
        return o
    if kind == "tail":        # rows before the first group and behind the last
        return np.sort(rng.integers(rows // 8, rows - rows // 8 + 1, groups + 1))
    return np.concatenate([[0], np.sort(rng.integers(0, rows + 1, groups - 1)), [rows]])


def weight(groups, out, inn, dtype, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    wide = (torch.randn(groups, out, inn + pad, generator=gen) * inn ** -0.5).to(dtype).cuda()
    return wide[:, :, :inn]


def routed_rows(offsets, rows):
    used = np.zeros(rows, bool)
    used[slice(0, rows) if offsets is None else slice(offsets[0], offsets[-1])] = True
    return used


# rows, in, out, groups, split, pad
LINEAR = [
    (1, 8, 8, 1, "layer", 0), (1, 1, 1, 1, "layer", 0), (3, 64, 16, 1, "layer", 0), (16, 2048, 40, 1, "layer", 0),
    (17, 136, 24, 4, "random", 0), (48, 512, 200, 16, "random", 8), (33, 72, 136, 3, "one", 0),
    (200, 264, 264, 1, "layer", 8), (300, 64, 512, 2, "random", 0), (129, 8, 129, 1, "layer", 0),
    (257, 200, 96, 5, "tail", 0), (400, 96, 320, 70, "random", 0), (64, 40, 24, 6, "empty", 0),
    (500, 77, 51, 3, "random", 0), (130, 129, 255, 1, "layer", 1), (260, 65, 9, 4, "tail", 3),
    (1100, 520, 136, 3, "random", 0), (2100, 72, 1032, 2, "tail", 0), (333, 98, 150, 3, "random", 2),
    (150, 6, 10, 2, "tail", 0), (700, 260, 12, 3, "random", 4), (20000, 34, 514, 90, "random", 0),
    (40000, 40, 136, 12, "random", 0), (40000, 33, 130, 12, "tail", 1),
]


def linear_case(rows, inn, out, groups, kind, pad, dtype, act, bias, residual, keep, seed=11):
    dt = DT[dtype]
    offsets = split(kind, rows, groups, seed)
    x, w = rows_of(rows, inn, dt, seed, pad), weight(groups, out, inn, dt, seed + 1, pad)
    b = rows_of(groups, out, dt, seed + 2) if bias else None
    res = rows_of(rows, out, dt, seed + 3, pad) if residual else None
    y, pre = rows_of(rows, out, dt, seed + 4, pad), rows_of(rows, out, dt, seed + 5, pad) if keep else None
    y0, pre0 = f64(y), f64(pre)
    off = None if offsets is None else torch.from_numpy(offsets.astype(np.int32)).cuda()
    if offsets is None and seed % 2:   # a layer's weight and bias without the groups' dimension
        got = D.linear(x, w[0], None if b is None else b[0], act, res, None, pre, y)
    else:
        got = D.linear(x, w, b, act, res, off, pre, y)
    assert got is y
    want, want_pre = O.linear(f64(x), f64(w), f64(b), act, f64(res), offsets, y0, pre0)
    used = routed_rows(offsets, rows)
    np.testing.assert_array_equal(f64(y)[~used], y0[~used])
    _, size = O.linear(np.abs(f64(x)), np.abs(f64(w)), None if b is None else np.abs(f64(b)), "none", None, offsets)
    _, z = O.linear(f64(x), f64(w), f64(b), "none", None, offsets)
    err = (inn + 4) * U * size
    if keep:
        np.testing.assert_array_equal(f64(pre)[~used], pre0[~used])
        within(pre[torch.from_numpy(used)], want_pre[used], (err + half(dt) * np.abs(z))[used], "pre")
    err = err * 1.2 + (32 * U * (1 + np.abs(z)) if act != "none" else 0) + 2 * U * np.abs(want)
    if residual:
        err = err + 2 * U * np.abs(f64(res))
    within(y[torch.from_numpy(used)], want[used], (err + half(dt) * np.abs(want))[used], "y")
    return y


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(map(str, c)))
def test_linear(case, dtype):
    announce(f"linear {case} {dtype}")
    linear_case(*case, dtype, "none", False, False, False, seed=12)
    linear_case(*case, dtype, "gelu_tanh", True, True, True, seed=13)


@gpu
@pytest.mark.parametrize("act", sorted(D.ACTIVATIONS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_activations(dtype, act):
    announce(f"linear {act} {dtype}")
    for bias, residual, keep in ((True, False, True), (False, True, False)):
        linear_case(150, 96, 72, 3, "random", 0, dtype, act, bias, residual, keep)
        linear_case(20, 96, 72, 3, "random", 0, dtype, act, bias, residual, keep)


@gpu
@pytest.mark.parametrize("rows,inn,out,groups", [(6000, 512, 768, 3), (9000, 64, 2048, 1), (2500, 1000, 1000, 40)])
def test_linear_large(rows, inn, out, groups):
    announce(f"linear {rows} x {inn} x {out}, {groups} groups")
    linear_case(rows, inn, out, groups, "layer" if groups == 1 else "random", 0, "bf16", "silu", True, True, True)


@gpu
@pytest.mark.parametrize("act", sorted(D.ACTIVATIONS))
def test_activations_far_out(act):
    """z far from zero and not finite: a unit weight hands it through."""
    announce(f"{act} far out")
    z = torch.tensor([0.0, -0.0, 1e-30, 5.0, -5.0, 30.0, -30.0, 90.0, -90.0, 1e4, -1e4, 1e12, -1e12, 1e30, -1e30])
    x = torch.zeros(len(z), 8)
    x[:, 0] = z
    w = torch.zeros(8, 8)
    w[0, 0] = 1.0
    y = f64(D.linear(x.cuda(), w.cuda(), activation=act))[:, 0]
    zz = f64(z)
    with np.errstate(over="ignore"):
        want = np.where(np.abs(zz) > 50, np.where((zz > 0) | (act == "none"), zz, 0.0), O.activation(act, np.clip(zz, -50, 50)))
    # values below the smallest float32 may be zero: 1e-37
    assert (np.abs(y - want) <= 32 * U * (1 + np.abs(zz)) * np.minimum(1, np.abs(want) + 1e-30) + 1e-37).all(), (y, want)
    dx = torch.zeros(len(z), 8, device="cuda")
    one = torch.zeros(len(z), 8)
    one[:, 0] = 1.0
    pre = x.cuda()
    D.linear_grad(one.cuda(), w=w.cuda(), activation=act, pre=pre, dx=dx)
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(np.abs(zz) > 50, np.where((zz > 0) | (act == "none"), 1.0, 0.0), O.slope(act, np.clip(zz, -50, 50)))
    assert (np.abs(f64(dx)[:, 0] - want) <= 64 * U * (1 + np.minimum(50, np.abs(zz)))).all(), (f64(dx)[:, 0], want)
    # NaN stays, infinity does not turn into another number
    x[0, 0], x[1, 0] = float("nan"), float("inf")
    y = D.linear(x.cuda(), w.cuda(), activation=act)[:, 0].cpu()
    assert torch.isnan(y[0])


@gpu
def test_infinite_values_stay_in_their_rows():
    """NaN and infinity in rows of another group, in rows of no group, and
    behind a row's end in a wider buffer reach no other row."""
    announce("rows of other groups with NaN")
    for dtype, pad in (("bf16", 8), ("bf16", 0), ("bf16", 5), ("f32", 4), ("f32", 1)):
        dt = DT[dtype]
        rows, inn, out, offsets = 90, 40, 48, [10, 30, 70, 80]
        wide = torch.full((rows, inn + pad), float("nan"), dtype=dt, device="cuda")
        x = wide[:, :inn]
        good = list(range(30, 70))
        x[30:70] = rows_of(40, inn, dt, 1)
        w = weight(3, out, inn, dt, 2, pad)
        w[0] = float("inf")
        w[2] = float("nan")
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        y = torch.zeros(rows, out, dtype=dt, device="cuda")
        D.linear(x, w, offsets=off, out=y)
        assert torch.isfinite(y[good]).all() and (y[:10] == 0).all() and (y[80:] == 0).all()
        dy = torch.full((rows, out + pad), float("inf"), dtype=dt, device="cuda")[:, :out]
        dy[30:70] = rows_of(40, out, dt, 3)
        dx, dw = torch.zeros(rows, inn, dtype=dt, device="cuda"), torch.zeros(3, out, inn, device="cuda")
        db = torch.zeros(3, out, device="cuda")
        D.linear_grad(dy, x, w, offsets=off, dx=dx, dw=dw, db=db)
        assert torch.isfinite(dx[good]).all() and torch.isfinite(dw[1]).all() and torch.isfinite(db[1]).all()
        want, want_w, want_b = O.linear_grad(f64(dy[30:70]), f64(x[30:70]), f64(w[1:2]))
        _, size_w, size_b = O.linear_grad(np.abs(f64(dy[30:70])), np.abs(f64(x[30:70])), np.abs(f64(w[1:2])))
        within(dw[1:2], want_w, 45 * U * size_w, "dw")
        within(db[1:2], want_b, 45 * U * size_b, "db")
        sx, _, _ = O.linear_grad(np.abs(f64(dy[30:70])), np.abs(f64(x[30:70])), np.abs(f64(w[1:2])))
        within(dx[30:70], want, 52 * U * sx + half(dt) * np.abs(want), "dx")


def grad_case(rows, inn, out, groups, kind, pad, dtype, grad_dtype, act, x_act, accumulate, seed=21, parts=("dx", "dw", "db")):
    dt, gt = DT[dtype], DT[grad_dtype]
    offsets = split(kind, rows, groups, seed)
    off = None if offsets is None else torch.from_numpy(offsets.astype(np.int32)).cuda()
    dy, x = rows_of(rows, out, dt, seed, pad), rows_of(rows, inn, dt, seed + 1, pad)
    w = weight(groups, out, inn, dt, seed + 2, pad)
    pre = rows_of(rows, out, dt, seed + 3, pad, 2.0) if act != "none" else None
    x_pre = rows_of(rows, inn, dt, seed + 4, pad, 2.0) if x_act != "none" else None
    dx = rows_of(rows, inn, dt, seed + 5, pad) if "dx" in parts else None
    dw = weight(groups, out, inn, gt, seed + 6, pad) if "dw" in parts else None
    db = rows_of(groups, out, gt, seed + 7) if "db" in parts else None
    dx0, dw0, db0 = f64(dx), f64(dw), f64(db)
    D.linear_grad(dy, x if dw is not None else None, w if dx is not None or dw is None else None, act, pre, off, dx, dw, db,
                  accumulate, x_act, x_pre)
    keep = (dw0, db0) if accumulate else (None, None)
    want, want_w, want_b = O.linear_grad(f64(dy), f64(x), f64(w), act, f64(pre), offsets, x_act, f64(x_pre), dx0, *keep)
    # sums of absolute values, and what the rounded dz moves
    z = np.zeros((rows, out)) if pre is None else f64(pre)
    slopes = np.abs(O.slope(act, z))
    dz, off_dz = np.abs(f64(dy)) * slopes, 0.0
    if act != "none":
        off_dz = np.abs(f64(dy)) * (64 * U * (1 + np.abs(z)) + (half(dt) + U) * slopes * (1 + half(dt)))
    ax, aw = np.abs(f64(x)), np.abs(f64(w))
    sx, sw, sb = O.linear_grad(dz, ax, aw, offsets=offsets)
    ex, ew, eb = O.linear_grad(np.broadcast_to(off_dz, dz.shape), ax, aw, offsets=offsets)
    n = rows if offsets is None else int(max(np.diff(offsets)))
    used = routed_rows(offsets, rows)
    if dx is not None:
        xz = np.zeros((rows, inn)) if x_pre is None else f64(x_pre)
        xs = np.abs(O.slope(x_act, xz))
        err = (1.01 * ex + (out + 4) * U * sx) * (xs + 1e-4) + (sx * 64 * U * (1 + np.abs(xz)) if x_act != "none" else 0)
        np.testing.assert_array_equal(f64(dx)[~used], dx0[~used])
        within(dx[torch.from_numpy(used)], want[used], (err + (U + half(dt)) * np.abs(want))[used], "dx")
    if dw is not None:
        old = np.abs(dw0) if accumulate else 0
        within(dw, want_w, 1.01 * ew + (n + 4) * U * sw + 2 * U * old + half(gt) * np.abs(want_w), "dw")
    if db is not None:
        old = np.abs(db0) if accumulate else 0
        within(db, want_b, 1.01 * eb + (n + 4) * U * sb + 2 * U * old + half(gt) * np.abs(want_b), "db")


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(map(str, c)))
def test_linear_grad(case, dtype):
    announce(f"linear_grad {case} {dtype}")
    grad_case(*case, dtype, "f32", "none", "none", False)
    grad_case(*case, dtype, "f32", "gelu_tanh", "silu", True)


@gpu
@pytest.mark.parametrize("act", sorted(D.ACTIVATIONS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_grad_activations(dtype, act):
    announce(f"linear_grad {act} {dtype}")
    grad_case(150, 96, 72, 3, "random", 0, dtype, "bf16", act, "none", False)
    grad_case(150, 96, 72, 3, "tail", 0, dtype, "bf16", "none", act, True)
    grad_case(75, 51, 33, 2, "random", 1, dtype, "f32", act, act, True)


@gpu
@pytest.mark.parametrize("parts", [("dx",), ("dw",), ("db",), ("dw", "db"), ("dx", "db")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_grad_of_some(dtype, parts):
    announce(f"linear_grad {parts} {dtype}")
    grad_case(200, 64, 40, 3, "random", 0, dtype, "f32", "silu", "none", True, parts=parts)
    grad_case(200, 64, 40, 1, "layer", 0, dtype, "bf16", "none", "none", False, parts=parts)


@gpu
@pytest.mark.parametrize("rows,inn,out,groups,kind", [(5000, 64, 72, 1, "layer"), (4100, 200, 136, 2, "random"),
                                                     (3000, 45, 77, 2, "tail"), (6000, 512, 768, 3, "random"),
                                                     (2500, 1000, 1000, 40, "random"), (4096, 128, 128, 4, "empty")])
def test_linear_grad_long(rows, inn, out, groups, kind):
    """Long groups, whose rows are split where the tiles are few."""
    announce(f"linear_grad {rows} x {inn} x {out}, {groups} groups, {kind}")
    grad_case(rows, inn, out, groups, kind, 0, "bf16", "f32", "silu", "none", True)
    grad_case(rows, inn, out, groups, kind, 0, "bf16", "bf16", "none", "none", False)
    if rows <= 5000:
        grad_case(rows, inn, out, groups, kind, 0, "f32", "f32", "none", "none", False)
