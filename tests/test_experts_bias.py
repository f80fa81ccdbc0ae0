"""The bias gradient sums dz = dy act'(pre) in float32, unrounded: dz is rounded
to the dtype only as an operand of the matrix units.

With U = 2^-24 and n rows in a group, db is off by (n + 4) U of the sum of the
|dz| (n terms and their products' rounding), by 64 U (1 + |z|) |dy| a term from
the slope, and by half a step of the stored type.  A bf16 dz would add 2^-9 of
each |dz| on average, about sqrt(n) 2^-9 |dz| in all, against n^2 U |dz| here:
for 200 rows twelve times the bound."""

import ctypes
import os

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from dimuon_newton_schulz_amd import experts as X
from oracle import expert_oracle as O
from test_experts import DT, U, announce, f64, half, rows_of, split, weight, within

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


@gpu
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows,out,groups,kind,pad", [(200, 40, 1, "layer", 0), (500, 72, 3, "random", 8), (90, 33, 2, "tail", 1),
                                                      (2000, 64, 1, "layer", 0), (64, 24, 5, "empty", 0), (1, 8, 1, "layer", 0)])
@pytest.mark.parametrize("parts", [("db",), ("dx", "dw", "db")])
def test_bias_gradient_of_unrounded_terms(rows, out, groups, kind, pad, act, parts):
    for dtype, grad_dtype, accumulate in (("bf16", "f32", False), ("bf16", "f32", True), ("f32", "f32", True), ("bf16", "bf16", False)):
        announce(f"db {rows} x {out}, {groups} groups {kind}, {act} {dtype} {grad_dtype} {accumulate} {parts}")
        dt, gt, inn = DT[dtype], DT[grad_dtype], 16
        offsets = split(kind, rows, groups, 3)
        off = None if offsets is None else torch.from_numpy(offsets.astype(np.int32)).cuda()
        dy, pre, x = rows_of(rows, out, dt, 1, pad), rows_of(rows, out, dt, 2, pad, 2.0), rows_of(rows, inn, dt, 3, pad)
        w = weight(groups, out, inn, dt, 4, pad)
        db = rows_of(groups, out, gt, 5)
        old = f64(db)
        dx, dw = (torch.zeros_like(x), torch.zeros(w.shape, dtype=gt, device="cuda")) if "dx" in parts else (None, None)
        D.linear_grad(dy, x, w, act, pre, off, dx, dw, db, accumulate)
        ones, none = np.ones((groups, out, 1)), np.zeros((rows, 1))
        _, _, want = O.linear_grad(f64(dy), none, ones, act, f64(pre), offsets, db=old if accumulate else None)
        _, _, size = O.linear_grad(np.abs(f64(dy) * O.slope(act, f64(pre))), none, ones, offsets=offsets)
        _, _, slopes = O.linear_grad(np.abs(f64(dy)) * 64 * U * (1 + np.abs(f64(pre))), none, ones, offsets=offsets)
        n = rows if offsets is None else int(max(np.diff(offsets)))
        bound = (n + 4) * U * size + slopes + 2 * U * (np.abs(old) if accumulate else 0) + half(gt) * np.abs(want)
        within(db, want, bound, "db")


@gpu
@pytest.mark.parametrize("rows,out,groups", [(70001, 24, 1), (9000, 130, 70), (3000, 257, 200), (17_000_000, 2, 1)])
def test_bias_gradient_of_many_tiles(rows, out, groups):
    """Tiles of rows of more than 64 groups, and more of them than workgroups
    at once; twice the same bits.  The reference is float64 on the GPU."""
    announce(f"db {rows} x {out}, {groups} groups")
    offsets = split("random", rows, groups, 7) if groups > 1 else np.array([5, rows - 3])
    off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dy, pre = (torch.randn(rows, out, generator=gen, device="cuda").bfloat16() for _ in range(2))
    got = []
    for _ in range(2):
        got.append(torch.full((groups, out), 9.0, device="cuda"))
        D.linear_grad(dy, activation="relu", pre=pre, offsets=off, db=got[-1])
    assert torch.equal(*got)
    dz = torch.where(pre > 0, dy.double(), 0.0)
    for g in range(groups):
        rs = slice(int(offsets[g]), int(offsets[g + 1]))
        want, size = dz[rs].sum(0), dz[rs].abs().sum(0)
        # (relu's slopes are exact)
        assert ((got[0][g].double() - want).abs() <= (rs.stop - rs.start + 4) * U * size + U * want.abs()).all(), g


@gpu
def test_bias_gradient_without_rows():
    announce("db of no rows")
    for accumulate, want in ((False, 0.0), (True, 3.0)):
        db = torch.full((8,), 3.0, device="cuda")
        e = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
        D.linear_grad(e, w=rows_of(8, 4, torch.bfloat16, 1), activation="silu", pre=e, db=db, accumulate=accumulate)
        assert (db == want).all()


@gpu
def test_bias_gradient_of_decreasing_offsets_touches_nothing_else():
    """The results are undefined; what lies behind the workspace and db is not written."""
    announce("db, decreasing offsets")
    rows, out, groups = 500, 72, 40
    dy, pre = rows_of(rows, out, torch.bfloat16, 1), rows_of(rows, out, torch.bfloat16, 2)
    off = torch.tensor([0, 500] * 20 + [0], dtype=torch.int32, device="cuda")   # 20 groups of all rows
    a = X.LinearGradArgs(rows=rows, in_=1, out=out, groups=groups, offsets=1, dtype=1, grad_dtype=0, activation=4, db=1)
    n = ctypes.c_size_t(0)
    assert D.load_library().linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    wide = torch.full((n.value + (1 << 16),), 77, dtype=torch.uint8, device="cuda")
    db = torch.full((groups + 8, out), 5.0, device="cuda")
    D.linear_grad(dy, activation="silu", pre=pre, offsets=off, db=db[4:groups + 4], workspace=wide[:n.value])
    assert (wide[n.value:] == 77).all() and (db[:4] == 5).all() and (db[-4:] == 5).all()


@built
def test_fewer_rows_need_no_larger_workspace():
    """linear_grad_workspace's tensor serves up to so many rows."""
    lib, n = D.load_library(), ctypes.c_size_t(0)
    for out, groups, act, dtype in ((8, 1, 4, 1), (768, 1, 4, 1), (1408, 64, 2, 1), (5000, 3, 1, 1), (768, 4, 4, 0), (768, 4, 0, 1)):
        before = 0
        for rows in [*range(0, 3000, 7), *range(3000, 300000, 641), 1 << 20, 1 << 24, (1 << 30) - 1]:
            a = X.LinearGradArgs(rows=rows, in_=64, out=out, groups=groups, offsets=1, dtype=dtype, grad_dtype=0, activation=act,
                                 dw=1, db=1)
            assert lib.linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
            assert n.value >= before, (rows, out, groups)
            before = n.value


@gpu
def test_bias_gradient_captured_and_on_two_streams():
    """Replays of a captured backward, with eager work between them, and two
    streams at once give the eager bits."""
    announce("db captured, on two streams")
    rows, inn, out, groups = 3000, 64, 136, 5
    off = torch.linspace(0, rows, groups + 1, device="cuda").int()
    dy, pre, x, w = (rows_of(rows, out, torch.bfloat16, 1), rows_of(rows, out, torch.bfloat16, 2),
                     rows_of(rows, inn, torch.bfloat16, 3), weight(groups, out, inn, torch.bfloat16, 4))

    def buffers():
        return torch.zeros_like(x), torch.zeros(groups, out, inn, device="cuda"), torch.zeros(groups, out, device="cuda")

    def backward(into, stream=None):
        D.linear_grad(dy, x, w, "gelu", pre, off, *into, accumulate=True, stream=stream)

    want = [buffers()]
    for _ in range(3):   # (each adds to what the one before left)
        want.append(tuple(t.clone() for t in want[-1]))
        backward(want[-1])
    into, eager = buffers(), buffers()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        backward(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        backward(into)
    for step in range(1, 4):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(into, want[step])), step
        backward(eager)
    two = [(buffers(), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in two:
            backward(b, s)
    torch.cuda.synchronize()
    for b, _ in two:
        assert all(torch.equal(a, t) for a, t in zip(b, want[3]))
