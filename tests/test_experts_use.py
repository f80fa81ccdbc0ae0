"""The experts' operators as a program uses them: an expert layer forward and
backward with its weight gradients read by Muon's plan, captured and replayed,
on other streams, at the ends of their ranges; and the products' machine code."""

import ctypes
import os
import sys
import threading

import numpy as np
import pytest
import torch

import dimuon_newton_schulz_amd as D
from dimuon_newton_schulz_amd import experts as X
from oracle import expert_oracle as O
from test_experts import U, f64, half, make_ids, rows_of, routed, weight, within
from test_kernel_code import OBJDUMP, kernels  # noqa: F401 (a fixture)

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


def announce(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


# ---------------------------------------------------------------------------
# An expert layer
# ---------------------------------------------------------------------------
class Layer:
    """x -> x + sum over a token's experts of weight * down(silu(up(x))), with
    buffers that stay where they are."""

    def __init__(self, tokens=200, top=2, experts=5, width=64, hidden=96, dtype=torch.float32, seed=1, drop=0.1):
        self.experts, self.dtype = experts, dtype
        self.ids = make_ids(tokens, top, experts, drop, seed, torch.int64).cuda()
        self.x, self.dy = rows_of(tokens, width, dtype, seed), rows_of(tokens, width, dtype, seed + 1)
        self.weights = torch.softmax(rows_of(tokens, top, torch.float32, seed + 2), 1)
        self.up, self.down = weight(experts, hidden, width, dtype, seed + 3), weight(experts, width, hidden, dtype, seed + 4)
        self.d_up, self.d_down = torch.zeros_like(self.up), torch.zeros_like(self.down)
        slots = tokens * top
        self.pre, self.h = (torch.zeros(slots, hidden, dtype=dtype, device="cuda") for _ in range(2))
        self.dh = torch.zeros_like(self.h)
        self.dxs = torch.zeros(slots, width, dtype=dtype, device="cuda")

    def forward(self):
        r = self.routes = D.expert_sort(self.ids, self.experts)
        self.xs = D.expert_gather(self.x, r)
        D.linear(self.xs, self.up, activation="silu", offsets=r.offsets, pre=self.pre, out=self.h)
        self.ys = D.linear(self.h, self.down, offsets=r.offsets)
        self.y = D.expert_combine(self.ys, r, self.weights, self.x)
        return self.y

    def backward(self):
        r = self.routes
        dys, self.dw = D.expert_combine_grad(self.dy, self.ys, self.weights, r)
        D.linear_grad(dys, self.h, self.down, offsets=r.offsets, dx=self.dh, dw=self.d_down, x_activation="silu",
                      x_pre=self.pre)
        D.linear_grad(self.dh, self.xs, self.up, offsets=r.offsets, dx=self.dxs, dw=self.d_up)
        self.dx = D.expert_combine(self.dxs, r, residual=self.dy)

    def outputs(self):
        return {"y": self.y, "dx": self.dx, "dw": self.dw, "d_up": self.d_up, "d_down": self.d_down,
                "up": self.up, "down": self.down}

    def reference(self):
        """y and gradients in 64 bits, from autograd on the CPU."""
        x, up, down, w = (t.detach().double().cpu().requires_grad_() for t in (self.x, self.up, self.down, self.weights))
        ids, y = self.ids.cpu(), x
        for j in range(ids.shape[1]):
            for e in range(self.experts):
                t = torch.nonzero(ids[:, j] == e).view(-1)
                out = torch.nn.functional.silu(x[t] @ up[e].T) @ down[e].T
                y = y.index_add(0, t, out * w[t, j, None])
        y.backward(self.dy.double().cpu())
        return {"y": y.detach(), "dx": x.grad, "dw": w.grad, "d_up": up.grad, "d_down": down.grad}

    def plan(self):
        params = [D.Param(w=w[e], g=g[e], mom=torch.zeros_like(w[e])) for w, g in
                  ((self.up, self.d_up), (self.down, self.d_down)) for e in range(self.experts)]
        return D.Plan(params, D.config_for(params, ns_dtype="f32" if self.dtype == torch.float32 else "bf16"), dimuon=False)


@gpu
def test_expert_layer_matches_autograd():
    """Six products in a row over K <= 200 terms each, in float32: each is off
    by (K + 4) U of its sum of absolute values, which for independent normal
    values is about sqrt(K) times its result: 6 * 204 * sqrt(200) U = 1.1e-3
    of the norm in the worst case."""
    announce("expert layer, float32")
    layer = Layer()
    layer.forward()
    layer.backward()
    want, got = layer.reference(), layer.outputs()
    for name, ref in want.items():
        err = np.linalg.norm(f64(got[name]) - ref.numpy()) / np.linalg.norm(ref.numpy())
        assert err < 1.1e-3, (name, err)
        assert err > 0


@gpu
def test_expert_layer_bf16_with_muon_step_captured():
    """Forward, backward and Muon's step: eager steps twice give the same bits,
    and so do replays of a captured step, with eager work in between."""
    announce("expert layer, bf16, captured")
    states = {}
    for how in ("eager", "again", "graph"):
        layer = Layer(dtype=torch.bfloat16, width=128, hidden=64)
        plan = layer.plan()

        def step():
            layer.forward()
            layer.backward()
            plan.step()

        if how == "graph":
            keep = {k: v.clone() for k, v in (("up", layer.up), ("down", layer.down))}
            moms = [p.mom for p in plan.params]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()   # first use outside the capture
            torch.cuda.current_stream().wait_stream(side)
            layer.up.copy_(keep["up"])
            layer.down.copy_(keep["down"])
            for m in moms:
                m.zero_()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            layer.up.copy_(keep["up"])
            layer.down.copy_(keep["down"])
            for m in moms:
                m.zero_()
            run = g.replay
        else:
            run = step
        trace = []
        for i in range(4):
            run()
            torch.cuda.synchronize()
            trace.append({k: v.clone() for k, v in layer.outputs().items()})
            other = Layer(tokens=50, seed=40 + i)   # eager work of the same kernels in between
            other.forward()
            other.backward()
        states[how] = trace
    for how in ("again", "graph"):
        for a, b in zip(states["eager"], states[how]):
            for k in a:
                assert torch.equal(a[k], b[k]), (how, k)
    assert not torch.equal(states["eager"][0]["up"], states["eager"][3]["up"])


@gpu
def test_gradient_accumulates_over_batches_in_flat_buffers():
    """dw and db of several batches in one float32 buffer, its views the
    gradients of a plan."""
    announce("accumulated gradients")
    experts, out, inn = 3, 40, 24
    flat = torch.zeros(experts * out * inn + 64, device="cuda")
    dw = flat[64:].view(experts, out, inn)
    want = np.zeros(dw.shape)
    size = np.zeros(dw.shape)
    for i in range(3):
        off = torch.tensor([0, 10 * i, 30, 50], dtype=torch.int32, device="cuda")
        dy, x = rows_of(50, out, torch.bfloat16, i), rows_of(50, inn, torch.bfloat16, 10 + i)
        D.linear_grad(dy, x, offsets=off, dw=dw, accumulate=True)
        _, want, _ = O.linear_grad(f64(dy), f64(x), np.zeros(dw.shape), offsets=off.cpu().numpy(), dw=want)
        _, size, _ = O.linear_grad(np.abs(f64(dy)), np.abs(f64(x)), np.zeros(dw.shape), offsets=off.cpu().numpy(), dw=size)
    within(dw, want, (50 + 8) * U * size, "dw")   # 50 terms an element in each of three sums, and two sums of those
    assert (flat[:64] == 0).all()


# ---------------------------------------------------------------------------
# Streams, threads, repeats
# ---------------------------------------------------------------------------
def layer_step(layer, stream=None):
    r = D.expert_sort(layer.ids, layer.experts, stream=stream)
    xs = D.expert_gather(layer.x, r, stream=stream)
    h = D.linear(xs, layer.up, activation="silu", offsets=r.offsets, pre=layer.pre, stream=stream)
    ys = D.linear(h, layer.down, offsets=r.offsets, stream=stream)
    y = D.expert_combine(ys, r, layer.weights, layer.x, stream=stream)
    dys, dw = D.expert_combine_grad(layer.dy, ys, layer.weights, r, stream=stream)
    D.linear_grad(dys, h, layer.down, activation="none", offsets=r.offsets, dx=layer.dh, dw=layer.d_down, stream=stream)
    D.linear_grad(layer.dh, xs, layer.up, activation="silu", pre=layer.pre, offsets=r.offsets, dx=layer.dxs,
                  dw=layer.d_up, stream=stream)
    n = int(r.offsets[-1]) if stream is None else None
    return r, y, dw, n


@gpu
def test_calls_on_given_streams_match_the_current_one():
    """With stream= every call takes the Python path; without, the native one.
    Both give the same bits, also for two layers on two streams at once."""
    announce("given streams")
    ref, two = [], []
    for seed in (3, 4):
        layer = Layer(dtype=torch.bfloat16, tokens=700, width=72, hidden=136, seed=seed)
        r, y, dw, n = layer_step(layer)
        ref.append([t.clone() for t in (r.offsets, r.order, r.place, y, dw, layer.d_up, layer.d_down, layer.dxs[:n])])
        layer.d_up.zero_(), layer.d_down.zero_(), layer.dxs.zero_()
        two.append((layer, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        results = [layer_step(layer, s) for layer, s in two]
        torch.cuda.synchronize()
        for want, (layer, _), (r, y, dw, _) in zip(ref, two, results):
            got = [r.offsets, r.order, r.place, y, dw, layer.d_up, layer.d_down, layer.dxs[:len(want[-1])]]
            for a, b in zip(want, got):
                assert torch.equal(a, b)


@gpu
def test_host_threads_call_at_once():
    announce("two host threads")
    layers = [Layer(dtype=torch.bfloat16, tokens=300, seed=s) for s in (5, 6)]
    want = [layer.forward().clone() for layer in layers]
    torch.cuda.synchronize()
    bad, streams = [], [torch.cuda.Stream() for _ in layers]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                y = layers[i].forward()
                if not torch.equal(y, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@gpu
@pytest.mark.parametrize("rows,inn,out,groups", [(3000, 512, 768, 5), (40, 2048, 200, 8), (700, 99, 130, 3)])
def test_products_repeat_bit_for_bit(rows, inn, out, groups):
    announce(f"repeats {rows} x {inn} x {out}, {groups} groups")
    off = torch.linspace(0, rows, groups + 1, device="cuda").int()
    x, w, dy = rows_of(rows, inn, torch.bfloat16, 1), weight(groups, out, inn, torch.bfloat16, 2), rows_of(rows, out, torch.bfloat16, 3)
    first = None
    for _ in range(10):
        y = D.linear(x, w, activation="gelu", offsets=off)
        dx, dw, db = torch.zeros_like(x), torch.zeros(groups, out, inn, device="cuda"), torch.zeros(groups, out, device="cuda")
        D.linear_grad(dy, x, w, offsets=off, dx=dx, dw=dw, db=db)
        got = [y, dx, dw, db]
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@gpu
def test_launch_events_name_the_calls():
    announce("launch events")
    layer = Layer(tokens=40)
    with D.LaunchTimer(16) as t:
        r = D.expert_sort(layer.ids, layer.experts)
        assert t.recorded() == 2 and D.LAUNCH_KINDS[t.kinds[1]] == "expert_sort"
        dz = torch.zeros(80, 96, device="cuda")
        db = torch.zeros(layer.experts, 96, device="cuda")
        D.linear_grad(dz, D.expert_gather(layer.x, r), layer.up, activation="silu", pre=layer.pre, offsets=r.offsets,
                      dx=layer.dxs, dw=layer.d_up, db=db)
        n = t.recorded()
        assert [D.LAUNCH_KINDS[k] for k in t.kinds[1:n]] == ["linear_slope", "linear_input", "linear_weight", "linear_bias"]


# ---------------------------------------------------------------------------
# Ends of the ranges
# ---------------------------------------------------------------------------
@gpu
def test_no_rows_and_no_tokens():
    announce("rows = 0, tokens = 0")
    e = torch.empty(0, 16, device="cuda")
    w = rows_of(8, 16, torch.float32, 1)
    assert D.linear(e, w).shape == (0, 8)
    dw, db = torch.ones(8, 16, device="cuda"), torch.ones(8, device="cuda")
    D.linear_grad(torch.empty(0, 8, device="cuda"), e, w, dx=e, dw=dw, db=db, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    D.linear_grad(torch.empty(0, 8, device="cuda"), e, w, activation="relu", pre=torch.empty(0, 8, device="cuda"), dx=e,
                  dw=dw, db=db)
    assert (dw == 0).all() and (db == 0).all()
    r = D.expert_sort(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4)
    assert r.offsets.tolist() == [0] * 5 and r.place.shape == (0, 3)
    xs = D.expert_gather(e, r)
    assert xs.shape == (0, 16) and D.expert_combine(xs, r).shape == (0, 16)


@gpu
def test_offsets_and_places_out_of_range_touch_nothing_else():
    """Offsets that are cut to the rows, places that count as unrouted."""
    announce("offsets and places out of range")
    x, w = rows_of(64, 32, torch.bfloat16, 1), weight(3, 16, 32, torch.bfloat16, 2)
    guard = torch.full((96, 16), 5.0, dtype=torch.bfloat16, device="cuda")
    y = guard[16:80]
    off = torch.tensor([-7, 20, 50, 10 ** 9], dtype=torch.int32, device="cuda")
    D.linear(x, w, offsets=off, out=y)
    want, _ = O.linear(f64(x), f64(w), offsets=[0, 20, 50, 64])
    size, _ = O.linear(np.abs(f64(x)), np.abs(f64(w)), offsets=[0, 20, 50, 64])
    within(y, want, 36 * U * size + 2.0 ** -8 * np.abs(want), "y")
    assert (guard[:16] == 5).all() and (guard[80:] == 5).all()
    dw = torch.zeros(3, 16, 32, device="cuda")
    D.linear_grad(y, x, offsets=off, dw=dw)
    _, want, _ = O.linear_grad(f64(y), f64(x), f64(w), offsets=[0, 20, 50, 64])
    _, size, _ = O.linear_grad(np.abs(f64(y)), np.abs(f64(x)), f64(w), offsets=[0, 20, 50, 64])
    within(dw, want, 68 * U * size, "dw")
    place = torch.tensor([[0, 10 ** 9], [-5, 1], [6, 2]], dtype=torch.int32, device="cuda")
    r = D.ExpertRoutes(torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda"), place)
    t = rows_of(3, 8, torch.float32, 3)
    xs = torch.zeros(6, 8, device="cuda")
    D.expert_gather(t, r, out=xs)
    assert torch.equal(xs[:3], t[[0, 1, 2]]) and (xs[3:] == 0).all()
    y = D.expert_combine(xs, r)
    assert torch.equal(y, t)


@gpu
def test_rows_behind_four_gigabytes():
    """Byte offsets of rows, weights and places beyond 32 bits."""
    announce("rows beyond 4 GiB")
    rows, inn, out, groups = 1_150_000, 2048, 16, 2
    x = torch.zeros(rows, inn, dtype=torch.bfloat16, device="cuda")
    tail = rows_of(300, inn, torch.bfloat16, 1)
    x[-300:] = tail
    w = weight(groups, out, inn, torch.bfloat16, 2)
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device="cuda")
    y = D.linear(x, w, offsets=off)
    want, _ = O.linear(f64(tail), f64(w), offsets=[0, 100, 300])
    size, _ = O.linear(np.abs(f64(tail)), np.abs(f64(w)), offsets=[0, 100, 300])
    within(y[-300:], want, (inn + 4) * U * size + 2.0 ** -8 * np.abs(want), "y")
    assert (y[:-300] == 0).all()
    dy = torch.zeros(rows, out, dtype=torch.bfloat16, device="cuda")
    dy[-300:] = rows_of(300, out, torch.bfloat16, 3)
    dx, dw = torch.zeros_like(x), torch.zeros(groups, out, inn, device="cuda")
    D.linear_grad(dy, x, w, offsets=off, dx=dx, dw=dw)
    want, want_w, _ = O.linear_grad(f64(dy[-300:]), f64(tail), f64(w), offsets=[0, 100, 300])
    size, size_w, _ = O.linear_grad(np.abs(f64(dy[-300:])), np.abs(f64(tail)), np.abs(f64(w)), offsets=[0, 100, 300])
    within(dx[-300:], want, 20 * U * size + 2.0 ** -8 * np.abs(want), "dx")
    within(dw, want_w, 304 * U * size_w, "dw")   # the other terms are exact zeros
    # one token in the last sorted row
    n = rows
    place = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    place[5, 0], place[n - 1, 0] = n - 1, 3
    order = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    order[n - 1], order[3] = 5, n - 1
    r = D.ExpertRoutes(torch.tensor([0, n], dtype=torch.int32, device="cuda"), order, place)
    D.expert_gather(x, r, out=dx)
    assert torch.equal(dx[3], tail[-1]) and (dx[n - 1] == 0).all()
    got = D.expert_combine(x, r)
    assert torch.equal(got[5], tail[-1]) and (got[:5] == 0).all() and (got[6:] == 0).all()


@gpu
def test_weights_behind_four_gigabytes():
    announce("weights beyond 4 GiB")
    groups, out, inn = 1100, 1024, 2048
    w = torch.zeros(groups, out, inn, dtype=torch.bfloat16, device="cuda")
    w[-1] = weight(1, out, inn, torch.bfloat16, 1)[0]
    for rows in (40, 5000):   # the kernel for few rows, and tiles
        x = rows_of(rows, inn, torch.bfloat16, 2)
        off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
        off[-1] = rows
        y = D.linear(x, w, offsets=off)
        ref = torch.nn.functional.linear(x.double(), w[-1].double())
        size = torch.nn.functional.linear(x.double().abs(), w[-1].double().abs())
        assert ((y.double() - ref).abs() <= (inn + 4) * U * size + 2.0 ** -8 * ref.abs()).all()
    dx, dy = torch.zeros_like(x), rows_of(rows, out, torch.bfloat16, 3)
    dw = torch.full_like(w, 3.0)
    D.linear_grad(dy, x, w, offsets=off, dx=dx, dw=dw)
    ref, size = dy.double() @ w[-1].double(), dy.double().abs() @ w[-1].double().abs()
    assert ((dx.double() - ref).abs() <= (out + 4) * U * size + 2.0 ** -8 * ref.abs()).all()
    ref, size = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    assert ((dw[-1].double() - ref).abs() <= (rows + 4) * U * size + 2.0 ** -8 * ref.abs()).all()
    assert (dw[:-1] == 0).all()


@gpu
def test_residual_in_place_and_columns_of_one_buffer():
    announce("in place")
    for rows, inn, out in ((9, 64, 40), (300, 72, 264), (1500, 64, 512)):
        wide = rows_of(rows, inn + out, torch.bfloat16, 1)
        x, y = wide[:, :inn], wide[:, inn:]
        keep = wide.clone()
        w = weight(1, out, inn, torch.bfloat16, 2)[0]
        D.linear(x, w, residual=y, out=y)
        want, _ = O.linear(f64(keep[:, :inn]), f64(w)[None], residual=f64(keep[:, inn:]))
        size, _ = O.linear(np.abs(f64(keep[:, :inn])), np.abs(f64(w))[None], residual=np.abs(f64(keep[:, inn:])))
        within(y, want, (inn + 6) * U * size + 2.0 ** -8 * np.abs(want), "y")
        assert torch.equal(x, keep[:, :inn])


@gpu
def test_native_and_python_marshalling_refuse_alike():
    """What is not the ordinary case goes on in Python, which says what is wrong."""
    announce("refusals with GPU tensors")
    x, w = rows_of(10, 16, torch.bfloat16, 1), rows_of(8, 16, torch.bfloat16, 2)
    r, _, _ = routed(5, 2, 4, 0.0)
    xs = rows_of(10, 16, torch.bfloat16, 3)
    bad = [
        lambda: D.linear(x, w.float()), lambda: D.linear(x, w, bias=rows_of(1, 8, torch.bfloat16, 3)),
        lambda: D.linear(x, w, residual=x), lambda: D.linear(x, w, out=x[:, :8]), lambda: D.linear(x[:, ::2], w[:, :8]),
        lambda: D.linear(x, w, offsets=r.offsets), lambda: D.linear(x.cpu(), w), lambda: D.linear(x, w.cpu()),
        lambda: D.linear(x, w, pre=rows_of(9, 8, torch.bfloat16, 3)),
        lambda: D.expert_sort(r.place.float(), 4), lambda: D.expert_sort(r.place, 0), lambda: D.expert_sort(r.place, 2000),
        lambda: D.expert_gather(rows_of(4, 16, torch.bfloat16, 1), r), lambda: D.expert_gather(xs.cpu(), r),
        lambda: D.expert_combine(xs, r, weights=rows_of(5, 3, torch.float32, 1)),
        lambda: D.expert_combine(xs, r, residual=xs), lambda: D.expert_combine(xs, r, out=xs[:5]),
        lambda: D.expert_combine_grad(rows_of(5, 16, torch.float32, 1), xs, rows_of(5, 2, torch.float32, 1), r),
        lambda: D.expert_combine_grad(xs[:5], xs, rows_of(5, 2, torch.float32, 1), r, dys=xs),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, D.MuonError)):
            call()
            pytest.fail(f"call {i} was not refused")


# ---------------------------------------------------------------------------
# Machine code
# ---------------------------------------------------------------------------
def stage_reads(code):
    """(16-byte reads, transposing reads) on every path from one barrier to the
    next that multiplies and reads fragments.  A path ends where the epilogue
    begins (it takes the accumulators out, turns or writes them)."""
    place = {address: i for i, (address, _, _) in enumerate(code)}
    counts, seen = set(), set()
    todo = [(i + 1, 0, 0, 0) for i, (_, text, _) in enumerate(code) if text.split()[0] == "s_barrier"]
    while todo:
        state = todo.pop()
        if state in seen or state[0] >= len(code):
            continue
        seen.add(state)
        at, wide, turned, mfma = state
        _, text, target = code[at]
        op = text.split()[0]
        if wide + turned > 64:   # (more than a stage has: the epilogue's loop, entered past its writes)
            continue
        if op == "s_barrier":
            if mfma and (wide or turned):
                counts.add((wide, turned))
            continue
        if op == "s_endpgm" or op.startswith(("ds_write", "v_permlane16_swap", "v_accvgpr_read", "buffer_store")):
            continue
        wide, turned, mfma = wide + (op == "ds_read_b128"), turned + (op == "ds_read_b64_tr_b16"), mfma + op.startswith("v_mfma")
        if op == "s_branch":
            todo.append((place[target], wide, turned, mfma))
            continue
        if op.startswith("s_cbranch"):
            todo.append((place[target], wide, turned, mfma))
        todo.append((at + 1, wide, turned, mfma))
    return counts


@built
@pytest.mark.skipif(not OBJDUMP, reason="llvm-objdump not installed")
def test_products_read_a_stage_between_its_barriers(kernels):  # noqa: F811
    """Each stage of a product's main loop reads the same number of fragments
    between its barriers, on every path (one number per tile shape of the
    kernel): none is read after the barrier that frees its buffer."""
    found = {name: code for name, code in kernels.items()
             if "k_linearILb0E" in name and any(i.startswith("v_mfma") for _, i, _ in code)}
    assert len(found) >= 10
    for name, code in found.items():
        counts = stage_reads(code)
        shapes = 3 if "GeoILi256ELi256E" in name else 1   # a full tile and two half ones
        assert 1 <= len(counts) <= shapes, (name, counts)
