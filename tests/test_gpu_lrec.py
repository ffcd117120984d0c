"""gdn_lrec_forward / _step / _backward on the GPU against the float64 oracle,
element by element, within the oracle's bound of a 32-bit evaluation's error
(oracle/block_oracle.py derives it) plus half a step of the output's type."""

import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_frame_amd import block
from gated_deltanet_recurrence_frame_amd import inputs as gin
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return gin.as_f64(t)


def close(got, ref, err, io, what):
    got = f64(got.cpu())
    assert got.shape == ref.shape
    tol = err + HALF[io] * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / tol))


def case(B, L, C, io, logits, seed=0, lengths=None):
    rng = np.random.Generator(np.random.PCG64(seed))
    z = 2.5 + 2.0 * rng.standard_normal((B, L, C))
    if not logits:
        z = 1.0 / (1.0 + np.exp(-z))
    c = {"x": rng.standard_normal((B, L, C)), "z": z, "d": rng.standard_normal((B, L, C))}
    c = {k: torch.from_numpy(v).to(DT[io]) for k, v in c.items()}
    c["h0"], c["dh"] = (torch.from_numpy(rng.standard_normal((B, C))).float() for _ in range(2))
    c["n"] = lengths
    return c


def on(t):
    return None if t is None else t.to(DEV)


def run(c, io, logits, complement, x=None, z=None):
    x = on(c["x"]) if x is None else x
    z = on(c["z"]) if z is None else z
    B, L, C = x.shape
    n = None if c["n"] is None else torch.tensor(c["n"], dtype=torch.int32, device=DEV)
    h0, dh, d = on(c["h0"]), on(c["dh"]), on(c["d"])
    plan = block.LrecPlan(B, L, C, io, DEV, logits, complement, saved=True, backward=True)
    o, h = plan.forward(x, z, h0, n)
    g = plan.backward(x, z, d, h0, dh, n, saved=plan.saved)
    g = {k: v.clone() for k, v in g.items()}
    g2 = plan.backward(x, z, d, h0, dh, n)
    torch.cuda.synchronize()
    a = [None if c[k] is None else f64(c[k]) for k in ("x", "z", "h0", "d", "dh")]
    (ro, rh), (eo, eh) = bo.lrec_forward(a[0], a[1], logits, complement, a[2], c["n"])
    close(o, ro, eo, io, "o")
    close(h, rh, eh, "fp32", "state")
    (dx, dz, dh0), (ex, ez, e0) = bo.lrec_backward(a[0], a[1], logits, complement, a[3], a[2],
                                                   a[4], c["n"])
    close(g["dx"], dx, ex, io, "dx")
    close(g["dgate"], dz, ez, io, "dgate")
    close(g["dstate_in"], dh0, e0, "fp32", "dstate_in")
    for k in g:      # without the saved buffer: the same states formed again
        assert torch.equal(g[k], g2[k]), k
    return o, h, g


SHAPES = [(1, 1, 1), (3, 1, 8), (1, 2, 3), (2, 15, 5), (1, 16, 256), (1, 17, 260), (2, 32, 40),
          (3, 33, 8), (2, 64, 36), (3, 65, 12), (2, 127, 12),
          (2, 128, 8), (1, 129, 64), (3, 300, 31), (1, 1000, 2), (2, 2177, 36), (1, 4500, 4)]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("logits", [True, False])
@pytest.mark.parametrize("complement", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, complement, logits, io):
    run(case(*shape, io, logits, seed=sum(shape)), io, logits, complement)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("logits", [True, False])
def test_without_states(logits, io):
    c = case(2, 200, 20, io, logits, seed=1)
    c["h0"] = c["dh"] = None
    run(c, io, logits, True)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [24, 33])
@pytest.mark.parametrize("complement", [True, False])
def test_padded_batch(complement, C, io):
    # every length at and around the edges of waves and chunks; NaN behind them
    L = 300
    lens = [L, 0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, L + 5, -2]
    eff = [min(max(n, 0), L) for n in lens]
    for logits in (True, False):
        c = case(len(lens), L, C, io, logits, seed=2, lengths=lens)
        for b, n in enumerate(eff):
            for k in ("x", "z", "d"):
                c[k][b, n:] = float("nan")
        dev = {k: on(c[k]) for k in ("x", "z")}
        for b, n in enumerate(eff):       # the oracle multiplies by a mask
            for k in ("x", "z", "d"):
                c[k][b, n:] = 0.0
        keep = c["d"].clone()
        for b, n in enumerate(eff):
            c["d"][b, n:] = float("nan")
        d_nan = c["d"]
        c["d"] = keep
        o, h, g = run(c, io, logits, complement, **dev)
        c["d"] = d_nan
        plan = block.LrecPlan(len(lens), L, C, io, DEV, logits, complement, backward=True)
        g2 = plan.backward(dev["x"], dev["z"], on(c["d"]), on(c["h0"]), on(c["dh"]),
                           torch.tensor(lens, dtype=torch.int32, device=DEV))
        for b, n in enumerate(eff):
            for t in (o, g["dx"], g["dgate"], g2["dx"], g2["dgate"]):
                assert not t[b, n:].any()
        for k in g2:
            assert bool(torch.isfinite(g2[k]).all()), k
        assert torch.equal(h[1], on(c["h0"])[1])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_gates_at_their_ends(io):
    # resets (a = 0) and held states (a = 1) inside chunks, at their edges
    B, L, C = 2, 400, 12
    c = case(B, L, C, io, True, seed=3)
    inf = float("inf")
    for t, v in ((0, -inf), (5, inf), (40, 88.0), (41, -88.0), (127, -inf), (128, -inf),
                 (200, inf), (201, -120.0), (202, 120.0), (255, -inf), (399, inf)):
        c["z"][:, t] = v
    run(c, io, True, True)
    run(c, io, True, False)
    c = case(B, L, C, io, False, seed=4)
    for t, v in ((0, 0.0), (64, 1.0), (127, 0.0), (128, 1.5), (129, -0.5), (300, 0.0)):
        c["z"][:, t] = v
    run(c, io, False, False)
    run(c, io, False, True)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [64, 35])
def test_inputs_out_of_a_projection(C, io):
    B, L = 3, 150
    c = case(B, L, C, io, True, seed=5)
    xz = torch.cat([c["x"], c["z"]], -1).to(DEV)
    o, h, g = run(c, io, True, True, x=xz[..., :C], z=xz[..., C:])
    plan = block.LrecPlan(B, L, C, io, DEV, True, True, backward=True)
    d = torch.full((B, L, 2 * C + 2), 7.0, dtype=DT[io], device=DEV)
    plan.backward(xz[..., :C], xz[..., C:], on(c["d"]), on(c["h0"]), on(c["dh"]),
                  dx=d[..., :C], dgate=d[..., C:2 * C])
    ref = plan.backward(xz[..., :C], xz[..., C:], on(c["d"]), on(c["h0"]), on(c["dh"]))
    assert torch.equal(d[..., :C], ref["dx"]) and torch.equal(d[..., C:2 * C], ref["dgate"])
    assert bool((d[..., 2 * C:] == 7.0).all())
    # token-major batches
    xt, zt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (xz[..., :C], xz[..., C:]))
    ot, ht = block.lrec_forward(xt, zt, on(c["h0"]), gate_logits=True, complement=True)
    assert torch.equal(ot, o) and torch.equal(ht, h)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_steps_and_windows_equal_one_call(io):
    B, L, C = 3, 150, 40
    c = case(B, L, C, io, True, seed=6)
    x, z, h0 = on(c["x"]), on(c["z"]), on(c["h0"])
    o, h = block.lrec_forward(x, z, h0, gate_logits=True, complement=True)
    plan = block.LrecPlan(B, 1, C, io, DEV, True, True)
    state, outs = h0.clone(), []
    for t in range(L):
        outs.append(plan.step(x[:, t:t + 1], z[:, t:t + 1], state).clone())
    (ro, rh), (eo, eh) = bo.lrec_forward(f64(c["x"]), f64(c["z"]), True, True, f64(c["h0"]))
    close(torch.cat(outs, 1), ro, eo, io, "steps")
    close(state, rh, eh, "fp32", "state of the steps")
    # windows, the state carried in place
    state, outs = h0.clone(), []
    for a, b in ((0, 1), (1, 64), (64, 150)):
        plan = block.LrecPlan(B, b - a, C, io, DEV, True, True)
        w, s = plan.forward(x[:, a:b], z[:, a:b], state, state_out=state)
        assert s is state
        outs.append(w)
    close(torch.cat(outs, 1), ro, eo, io, "windows")
    close(state, rh, eh, "fp32", "state of the windows")


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("B,L,C", [(40, 1, 700), (8, 16, 700), (8, 100, 700), (4, 129, 1400),
                                   (4, 900, 1400), (2, 3000, 1400)])
def test_state_in_place_equals_state_apart(B, L, C, io):
    # the last chunk writes its state over the one that the first chunks read
    c = case(B, L, C, io, True, seed=14)
    x, z, h0 = on(c["x"]), on(c["z"]), on(c["h0"])
    plan = block.LrecPlan(B, L, C, io, DEV, True, True)
    o, h = plan.forward(x, z, h0)
    o, h = o.clone(), h.clone()
    for _ in range(10):
        state = h0.clone()
        o2, _ = plan.forward(x, z, state, state_out=state)
        assert torch.equal(o2, o) and torch.equal(state, h)


def test_same_bits_every_time_on_any_stream():
    B, L, C = 2, 5000, 700
    c = case(B, L, C, "bf16", True, seed=7)
    x, z, d, h0, dh = (on(c[k]) for k in ("x", "z", "d", "h0", "dh"))

    def once():
        plan = block.LrecPlan(B, L, C, "bf16", DEV, True, True, saved=True, backward=True)
        o, h = plan.forward(x, z, h0)
        return [o, h, *plan.backward(x, z, d, h0, dh, saved=plan.saved).values()]

    first = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = once()
        third = once()
    side.synchronize()
    for a, b, e in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, e)


@pytest.mark.parametrize("L", [1, 100, 3000])
def test_captured_and_replayed(L):
    B, C = 2, 260
    c = case(B, L, C, "bf16", True, seed=8)
    x, z, d, h0, dh = (on(c[k]) for k in ("x", "z", "d", "h0", "dh"))
    plan = block.LrecPlan(B, L, C, "bf16", DEV, True, True, saved=True, backward=True)

    def once():
        o, h = plan.forward(x, z, h0)
        return [o, h, *plan.backward(x, z, d, h0, dh, saved=plan.saved).values()]

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = once()
    for i in range(4):
        x.mul_(1.125)
        h0.add_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = once()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_plans_on_two_streams_at_once():
    c = [case(1, 4000, 512, "bf16", True, seed=9 + i) for i in range(2)]
    data = [[on(k[n]) for n in ("x", "z", "d", "h0", "dh")] for k in c]
    plans = [block.LrecPlan(1, 4000, 512, "bf16", DEV, True, True, saved=True, backward=True)
             for _ in range(2)]

    def once(i):
        x, z, d, h0, dh = data[i]
        o, h = plans[i].forward(x, z, h0)
        return [o, h, *plans[i].backward(x, z, d, h0, dh, saved=plans[i].saved).values()]

    want = [[t.clone() for t in once(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(once(i))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)
