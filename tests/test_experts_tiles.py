"""The products' kernels by their tile: sizes that each of the larger tiles is
chosen for, with whole and partial last tiles in both directions, against
float64 products on the GPU, twice with the same bits.  The kernel that ran is
asserted, so that another choice of tiles does not leave one untested.

Bounds as in test_experts: (K + 4) U of the sum of absolute values, half a step
of the stored type, and what an activation or slope adds."""

import re

import numpy as np
import pytest
import torch
from torch.profiler import ProfilerActivity, profile

import dimuon_newton_schulz_amd as D
from test_experts import DT, U, announce, half

gpu = pytest.mark.gpu

NAME = re.compile(r"k_linear<(true|false), (\d), .*?Geo<(\d+), (\d+),.*?>, (\d+), (true|false)>")


def tiles(call):
    """(mode, rows, columns, alignment, plain) of the product kernels that a call launches; None where the profiler sees none."""
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    found = [NAME.search(e.name) for e in prof.events()]
    found = {(int(m[2]), int(m[3]), int(m[4]), int(m[5]), m[6] == "true") for m in found if m}
    return found or None


def data(rows, columns, dtype, seed, pad=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, columns + pad, generator=gen, device="cuda") * scale).to(dtype)[:, :columns]


def logistic(z, slope):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s)) if slope else z * s


def near(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(err).all() and (err <= bound).all(), (what, float((err - bound).max()), float(err.max()))


class Case:
    def __init__(self, rows, inn, out, groups, dtype, pad=0, seed=1):
        self.rows, self.inn, self.out, self.groups, self.dt = rows, inn, out, groups, DT[dtype]
        rng = np.random.default_rng(seed)
        self.bounds = [0, rows]
        self.off = None
        if groups > 1:   # rows before the first group and behind the last, one empty group
            inner = np.sort(rng.integers(rows // 10, rows - rows // 10, groups - 1))
            inner[groups // 2] = inner[groups // 2 - 1]
            self.bounds = [3, *map(int, inner), rows - 2]
            self.off = torch.tensor(self.bounds, dtype=torch.int32, device="cuda")
        self.x, self.dy = data(rows, inn, self.dt, 1, pad), data(rows, out, self.dt, 2, pad)
        self.w = data(groups * out, inn, self.dt, 3, scale=inn ** -0.5).view(groups, out, inn)

    def used(self):
        return slice(self.bounds[0], self.bounds[-1])

    def each(self):
        return [(g, slice(self.bounds[g], self.bounds[g + 1])) for g in range(self.groups)]

    def per_group(self, f, columns):
        """Rows of every group through f(rows, group)."""
        out = torch.zeros(self.rows, columns, dtype=torch.float64, device="cuda")
        for g, r in self.each():
            if r.start < r.stop:
                out[r] = f(r, g)
        return out


def forward(c, full):
    y, pre = (torch.full((c.rows, c.out), 3.0, dtype=c.dt, device="cuda") for _ in range(2))
    bias, res = (data(c.groups, c.out, c.dt, 4), data(c.rows, c.out, c.dt, 5)) if full else (None, None)
    kw = dict(bias=bias if c.groups > 1 or not full else bias[0], activation="silu", pre=pre) if full else {}
    w = c.w if c.groups > 1 else c.w[0]

    def call():
        if full:
            y.copy_(res)   # the residual in place
        return D.linear(c.x, w, offsets=c.off, residual=y if full else None, out=y, **kw)

    seen = tiles(call)
    first = y.clone()
    call()
    assert torch.equal(first, y)
    z = c.per_group(lambda r, g: c.x[r].double() @ c.w[g].double().t() + (bias[g].double() if full else 0), c.out)
    size = c.per_group(lambda r, g: c.x[r].double().abs() @ c.w[g].double().abs().t() + (bias[g].double().abs() if full else 0), c.out)
    err, u = (c.inn + 4) * U * size, c.used()
    if full:
        near(pre[u], z[u], (err + half(c.dt) * z.abs())[u], "pre")
        want = logistic(z, False) + res.double()
        err = err * 1.2 + 32 * U * (1 + z.abs()) + 2 * U * want.abs() + 2 * U * res.double().abs()
    else:
        want = z
    near(y[u], want[u], (err + (half(c.dt) + 2 * U) * want.abs())[u], "y")
    for r in (slice(0, u.start), slice(u.stop, c.rows)):
        assert torch.equal(y[r], res[r] if full else torch.full_like(y[r], 3.0)) and (pre[r] == 3).all()
    return seen


def input_gradient(c, full):
    dx = torch.full((c.rows, c.inn), 3.0, dtype=c.dt, device="cuda")
    x_pre = data(c.rows, c.inn, c.dt, 6, scale=2.0) if full else None
    w = c.w if c.groups > 1 else c.w[0]

    def call():
        return D.linear_grad(c.dy, w=w, offsets=c.off, dx=dx, x_activation="silu" if full else "none", x_pre=x_pre)

    seen = tiles(call)
    first = dx.clone()
    call()
    assert torch.equal(first, dx)
    want = c.per_group(lambda r, g: c.dy[r].double() @ c.w[g].double(), c.inn)
    size = c.per_group(lambda r, g: c.dy[r].double().abs() @ c.w[g].double().abs(), c.inn)
    err, u = (c.out + 4) * U * size, c.used()
    if full:
        z = x_pre.double()
        s = logistic(z, True)
        want, err = want * s, err * (s.abs() + 1e-4) + size * 64 * U * (1 + z.abs())
    near(dx[u], want[u], (err + (half(c.dt) + U) * want.abs())[u], "dx")
    assert (dx[:u.start] == 3).all() and (dx[u.stop:] == 3).all()
    return seen


def weight_gradient(c, accumulate, grad_dtype):
    gt = DT[grad_dtype]
    old = data(c.groups * c.out, c.inn, gt, 7).view(c.groups, c.out, c.inn)
    dw = old.clone()

    def call():
        dw.copy_(old)
        return D.linear_grad(c.dy, c.x, offsets=c.off, dw=dw if c.groups > 1 else dw[0], accumulate=accumulate)

    seen = tiles(call)
    first = dw.clone()
    call()
    assert torch.equal(first, dw)
    for g, r in c.each():
        want, size = c.dy[r].double().t() @ c.x[r].double(), c.dy[r].double().abs().t() @ c.x[r].double().abs()
        err = (r.stop - r.start + 4) * U * size
        if accumulate:
            want, err = want + old[g].double(), err + 2 * U * old[g].double().abs()
        near(dw[g], want, err + half(gt) * want.abs(), f"dw[{g}]")
    return seen


def check(seen, mode, shape, align, plain):
    if seen is not None:
        assert seen == {(mode, *shape, align, plain)}, seen


LARGE = (256, 256)
# rows, in, out, groups: last tiles of at most 128 rows and columns, and of more
FORWARD = [(3900, 1024, 3848, 1), (3990, 1032, 3976, 1), (3850, 1048, 3970 // 8 * 8, 1), (20000, 1544, 1288, 9)]


@gpu
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("rows,inn,out,groups", FORWARD)
def test_large_forward(rows, inn, out, groups, full):
    announce(f"forward {rows} x {inn} x {out}, {groups} groups, {'full' if full else 'plain'}")
    check(forward(Case(rows, inn, out, groups, "bf16", pad=8), full), 0, LARGE, 16, not full)


@gpu
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("rows,inn,out,groups", [(r, o, i, g) for r, i, o, g in FORWARD])
def test_large_input_gradient(rows, inn, out, groups, full):
    announce(f"input gradient {rows} x {inn} x {out}, {groups} groups, {'full' if full else 'plain'}")
    check(input_gradient(Case(rows, inn, out, groups, "bf16", pad=8), full), 1, LARGE, 16, not full)


@gpu
@pytest.mark.parametrize("accumulate,grad_dtype", [(False, "f32"), (False, "bf16"), (True, "f32"), (True, "bf16")])
@pytest.mark.parametrize("rows,inn,out,groups", [(1024, 3848, 3900 // 8 * 8, 1), (1100, 3976, 3992, 1), (48000, 1100 // 8 * 8, 1032, 20)])
def test_large_weight_gradient(rows, inn, out, groups, accumulate, grad_dtype):
    announce(f"weight gradient {rows} x {inn} x {out}, {groups} groups, {grad_dtype} {'added' if accumulate else ''}")
    check(weight_gradient(Case(rows, inn, out, groups, "bf16", pad=8), accumulate, grad_dtype), 2, LARGE, 16, not accumulate)


@gpu
@pytest.mark.parametrize("dtype,extra,align", [("bf16", 2, 4), ("f32", 0, 16), ("f32", 3, 4), ("bf16", 0, 16)])
def test_medium_tiles(dtype, extra, align):
    """More than 512 tiles of 128 x 128, with too little k for the large ones."""
    announce(f"medium tiles {dtype}, alignment {align}")
    c = Case(2970 + extra, 2952 + extra, 256 + extra, 1, dtype)
    for full in (False, True):
        check(input_gradient(c, full), 1, (128, 128), align, False)
    c = Case(300, 2952 + extra, 2960 + extra, 1, dtype)
    for accumulate in (False, True):
        check(weight_gradient(c, accumulate, "f32"), 2, (128, 128), align, False)
    c = Case(2970 + extra, 256 + extra, 2960 + extra, 1, dtype)
    for full in (False, True):
        check(forward(c, full), 0, (128, 128), align, False)
