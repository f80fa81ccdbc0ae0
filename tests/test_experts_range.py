"""Activations and slopes far out and where numbers are not finite, in both
types and on every path that forms one; weights beyond 4 GiB in tiles.

A unit weight hands z and the slope through.  In bf16 a slope is off by its own
rounding, 2^-8 of it, and 64 U (1 + |z|) as in float32 (slopes are cut to
|z| <= 100, and 0 or 1 beyond 50 to within U)."""

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from oracle import expert_oracle as O
from test_experts import DT, U, announce, f64, half, rows_of, weight
from test_experts_tiles import tiles

gpu = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
VALUES = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 5.0, -5.0, 12.0, -12.0, 30.0, -30.0, 90.0, -90.0, 101.0, -101.0, 1e4, -1e4, 1e12,
          -1e12, 1e19, -1e19, 1e30, -1e30, 3e38, -3e38, INF, -INF, NAN]


def slopes(act, z):
    """Of finite z and of infinities; NaN where z is."""
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.where(np.abs(z) > 50, ((z > 0) | (act == "none")).astype(float), O.slope(act, np.clip(z, -50, 50)))
    return np.where(np.isnan(z), 1.0 if act == "none" else NAN, s)


def alike(got, want, bound, what):
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all(), (what, got, want)
    assert (np.abs(got - want)[~nan] <= bound[~nan]).all(), (what, got, want)


@gpu
@pytest.mark.parametrize("act", sorted(D.ACTIVATIONS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations_far_out_in_both_types(dtype, act):
    """Rows in one group for the kernel of few rows, and many of them for tiles."""
    dt = DT[dtype]
    for copies in (1, 60):
        announce(f"{act} {dtype} far out, {copies} copies")
        x = torch.zeros(len(VALUES) * copies, 8, dtype=dt)
        x[:, 0] = torch.tensor(VALUES * copies).to(dt)
        w = torch.zeros(8, 8, dtype=dt)
        w[0, 0] = 1.0
        pre = torch.zeros(len(x), 8, dtype=dt, device="cuda")
        y = f64(D.linear(x.cuda(), w.cuda(), activation=act, pre=pre))[:, 0]
        z = f64(x)[:, 0]
        np.testing.assert_array_equal(f64(pre)[:, 0], z)
        low = z == -INF   # z times 0: no number, or the limit
        finite = np.isfinite(z)
        assert (y[z == INF] == INF).all() and np.isnan(y[np.isnan(z)]).all()
        assert ((y[low] == (-INF if act == "none" else 0)) | (np.isnan(y[low]) & (act not in ("none", "relu")))).all(), y[low]
        with np.errstate(over="ignore", invalid="ignore"):
            want = np.where(np.abs(z) > 50, np.where((z > 0) | (act == "none"), z, 0.0), O.activation(act, np.clip(z, -50, 50)))
        y, z, want = y[finite], z[finite], want[finite]
        # (1e-37: values below the least normal number may be zero)
        bound = 32 * U * (1 + np.abs(z)) * np.minimum(1, np.abs(want)) + half(dt) * np.abs(want) + 1e-37
        assert (np.abs(y - want) <= bound).all(), (y, want)


@gpu
@pytest.mark.parametrize("act", sorted(D.ACTIVATIONS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slopes_far_out_on_every_path(dtype, act):
    """dz in dx, in dw and in db, and the slope of the activation that made x."""
    announce(f"slopes of {act} {dtype} far out")
    dt, n = DT[dtype], len(VALUES)
    z = torch.zeros(n, 8, dtype=dt)
    z[:, 0] = torch.tensor(VALUES).to(dt)
    one = torch.zeros(n, 8, dtype=dt)
    one[:, 0] = 1.0
    eye = torch.eye(8, dtype=dt).expand(n, 8, 8).contiguous().cuda()
    off = torch.arange(n + 1, dtype=torch.int32, device="cuda")   # a group per row
    pre, dy = z.cuda(), one.cuda()
    want = slopes(act, f64(z)[:, 0])
    of_slope = 64 * U * (1 + np.minimum(50, np.abs(np.nan_to_num(f64(z)[:, 0]))))
    bound = of_slope + half(dt) * np.abs(want)
    dx, dw, db = torch.zeros(n, 8, dtype=dt, device="cuda"), torch.zeros(n, 8, 8, device="cuda"), torch.zeros(n, 8, device="cuda")
    D.linear_grad(dy, dy, eye, act, pre, off, dx, dw, db)
    alike(f64(dx)[:, 0], want, bound, "dx")
    alike(f64(dw)[:, 0, 0], want, bound, "dw")
    alike(f64(db)[:, 0], want, of_slope, "db")
    alone = torch.zeros_like(db)
    D.linear_grad(dy, w=eye, activation=act, pre=pre, offsets=off, db=alone)
    alike(f64(alone)[:, 0], want, of_slope, "db alone")
    # rows by element: a width that is no multiple of eight, and one that is odd
    for columns in (6, 7):
        got = torch.zeros(n, columns, device="cuda")
        D.linear_grad(dy[:, :columns].contiguous(), activation=act, pre=pre[:, :columns].contiguous(), offsets=off, db=got)
        alike(f64(got)[:, 0], want, of_slope, f"db of {columns}")
    dx = torch.zeros(n, 8, dtype=dt, device="cuda")
    D.linear_grad(dy, w=eye[0], dx=dx, x_activation=act, x_pre=pre)
    alike(f64(dx)[:, 0], want, bound, "dx through x_pre")
    # x_pre of 60 copies: tiles
    many = torch.zeros(60 * n, 8, dtype=dt, device="cuda")
    D.linear_grad(dy.repeat(60, 1), w=eye[0], dx=many, x_activation=act, x_pre=pre.repeat(60, 1))
    assert torch.equal(torch.nan_to_num(many.view(60, n, 8)[:, :, 0], 7.0), torch.nan_to_num(dx[:, 0], 7.0).expand(60, n))


@gpu
def test_tiles_of_weights_behind_four_gigabytes():
    """Enough rows that the last group's are taken in tiles."""
    announce("tiles of weights beyond 4 GiB")
    groups, out, inn, rows = 1100, 1024, 2048, 50000
    w = torch.zeros(groups, out, inn, dtype=torch.bfloat16, device="cuda")
    w[-1] = weight(1, out, inn, torch.bfloat16, 1)[0]
    x = rows_of(rows, inn, torch.bfloat16, 2)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[-1] = rows
    y = torch.empty(rows, out, dtype=torch.bfloat16, device="cuda")
    seen = tiles(lambda: D.linear(x, w, offsets=off, out=y))
    assert seen is None or {s[0] for s in seen} == {0}, seen
    some = torch.arange(0, rows, 7, device="cuda")
    a, b = x[some].double(), w[-1].double().t().contiguous()
    want, size = a @ b, a.abs() @ b.abs()
    assert ((y[some].double() - want).abs() <= (inn + 4) * U * size + 2.0 ** -8 * want.abs()).all()
