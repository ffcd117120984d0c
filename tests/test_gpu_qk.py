"""gdn_qk_forward / gdn_qk_backward and the 8-bit checkpoints on the GPU
against the float64 oracle, element by element.

Tolerances, with u = 2^-24 and the oracle's magnitudes m (the formula with
absolute values): an output of the io type is off by at most half a step of
its own rounding plus K u m.
  forward   r: a lane's at most 16 squares in turn and 6 tree sums, halved by
            the root, eps, root and division: 13 u; times x and w: 2 u; cosine
            and sine: 4 u of their own and pi u of the reduced angle; products
            and sum 3 u.  Below 26 u: K = 32.
  dx        g 12 u, w, r and the difference: 28 u; the other term r x (14 u) by
            the dot product (14 + 13 + 22 u), c, product and r: 81 u.  K = 96.
  dw        a term 27 u, then at most one rounding per row summed (R rows).
"""

import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_frame_amd import block
from gated_deltanet_recurrence_frame_amd import inputs as gin
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return gin.as_f64(t)


def close(got, ref, err, io):
    """|got - ref| within err, rounded to io."""
    got = f64(got)
    assert got.shape == ref.shape
    tol = err + HALF[io] * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%d of %d off, worst %.3g of its tolerance" % (
        bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / tol))


def rows(rng, shape, io):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)))
    return torch.from_numpy(x).to(DT[io])


def case(B, L, Hq, Hk, D, pairs, io, weights=True, seed=0, top=4000):
    rng = np.random.Generator(np.random.PCG64(seed))
    c = {"q": rows(rng, (B, L, Hq, D), io), "k": rows(rng, (B, L, Hk, D), io),
         "dy": [rows(rng, (B, L, h, D), io) for h in (Hq, Hk)],
         "positions": None, "wq": None, "wk": None}
    if pairs:
        c["positions"] = torch.from_numpy(
            rng.integers(-top, top, (B, L, len(pairs)))).to(torch.int32)
    if weights:
        c["wq"], c["wk"] = (torch.from_numpy(1 + 0.5 * rng.standard_normal(D)).float()
                            for _ in range(2))
    return c


def phi_of(c, pairs, theta):
    return bo.qk_angles(c["positions"].numpy(), pairs, theta) if pairs else None


def on(t):
    return None if t is None else t.to(DEV)


def run(c, pairs, io, norm, eps, pairing, theta=10000.0, extra=0.0, q=None, k=None):
    """Forward and backward of a case against the oracle."""
    q = on(c["q"]) if q is None else q
    k = on(c["k"]) if k is None else k
    kw = dict(norm=norm, eps=eps, axis_pairs=pairs, pairing=pairing, theta=theta)
    rest = (on(c["positions"]), on(c["wq"]), on(c["wk"]))
    yq, yk = block.qk_forward(q, k, *rest, **kw)
    g = block.qk_backward(on(c["dy"][0]), on(c["dy"][1]), q, k, *rest, **kw)
    torch.cuda.synchronize()
    phi = phi_of(c, pairs, theta)
    for y, n, w, dy in ((yq, "q", c["wq"], c["dy"][0]), (yk, "k", c["wk"], c["dy"][1])):
        wv = None if w is None else f64(w)
        ref, mag = bo.qk_forward(f64(c[n]), wv, phi, norm, eps, pairing)
        close(y.cpu(), ref, (32 * U + extra) * mag, io)
        (dx, dw), (dxm, dwm) = bo.qk_backward(f64(c[n]), wv, phi, norm, eps, pairing, f64(dy))
        close(g["d" + n].cpu(), dx, (96 * U + 3 * extra) * dxm, io)
        R = dy.shape[0] * dy.shape[1] * dy.shape[2]
        if w is not None:
            close(g["d%s_weight" % n].cpu(), dw, ((32 + R) * U + extra) * dwm, "fp32")
        else:
            assert "d%s_weight" % n not in g
    return yq, yk, g


SHAPES = [
    (1, 1, 1, 1, 4, (2,)),               # the smallest
    (2, 5, 3, 1, 16, (4,)),
    (1, 37, 20, 20, 112, (16, 20, 20)),  # the mixer's heads, three axes
    (3, 9, 5, 2, 72, (18,)),             # pieces of 2 elements, 18 lanes a row
    (2, 3, 2, 2, 256, (128,)),           # whole head turned, largest head
    (1, 11, 4, 1, 96, (24,)),            # half of the head turned
    (2, 7, 9, 3, 48, (2, 6, 4)),
    (1, 300, 2, 1, 20, (2, 2)),          # 5 pieces of 4
    (1, 6, 3, 2, 64, ()),                # no rotation
]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rms_with_weights(shape, pairing, io):
    c = case(*shape, io)
    run(c, shape[5], io, "rms", 1e-6, pairing)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,eps", [("none", 0.0), ("l2", 0.0), ("l2", 1e-3), ("rms", 0.0)])
def test_norms_without_weights(norm, eps, io):
    shape = (2, 13, 5, 3, 80, (8, 16))
    c = case(*shape, io, weights=False, seed=1)
    run(c, shape[5], io, norm, eps, "halves")


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_one_operand_weighted(io):
    shape = (1, 13, 5, 3, 80, (8, 16))
    c = case(*shape, io, seed=2)
    c["wk"] = None
    run(c, shape[5], io, "rms", 1e-6, "adjacent")


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_far_positions(io):
    # positions up to 2^30: the product with a frequency is rounded to 2^-53
    # of at most 2^30 / 2 pi turns, 2^-23 radians on either side
    shape = (2, 33, 2, 2, 64, (16, 16))
    c = case(*shape, io, seed=3, top=2 ** 30)
    run(c, shape[5], io, "rms", 1e-6, "halves", theta=1e6, extra=2 * 2.0 ** -22)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_rows_out_of_a_projection(io):
    # q, k as slices of [B, L, (Hq + 2 Hk) D], and the gradients into one
    B, L, Hq, Hk, D, pairs = 3, 19, 6, 2, 112, (56,)
    c = case(B, L, Hq, Hk, D, pairs, io, seed=4)
    H = Hq + 2 * Hk
    qkv = torch.full((B, L, H, D), float("nan"), dtype=DT[io])
    qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk] = c["q"], c["k"]
    qkv = qkv.to(DEV)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    yq, yk, g = run(c, pairs, io, "rms", 1e-6, "halves", q=q, k=k)
    d = torch.full((B, L, H, D), 7.0, dtype=DT[io], device=DEV)
    block.qk_backward(on(c["dy"][0]), on(c["dy"][1]), q, k, on(c["positions"]), on(c["wq"]),
                      on(c["wk"]), axis_pairs=pairs, dq=d[:, :, :Hq], dk=d[:, :, Hq:Hq + Hk])
    torch.cuda.synchronize()
    assert torch.equal(d[:, :, :Hq], g["dq"]) and torch.equal(d[:, :, Hq:Hq + Hk], g["dk"])
    assert bool((d[:, :, Hq + Hk:] == 7.0).all())      # the values' part is left as it was
    # token-major batches, and a batch repeated by a stride of 0
    qt, kt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k))
    yt = block.qk_forward(qt, kt, on(c["positions"]), on(c["wq"]), on(c["wk"]), axis_pairs=pairs)
    assert torch.equal(yt[0], yq) and torch.equal(yt[1], yk)
    q1 = q[:1].expand(B, L, Hq, D)
    y1 = block.qk_forward(q1, k, on(c["positions"]), on(c["wq"]), on(c["wk"]), axis_pairs=pairs)
    y2 = block.qk_forward(q1.contiguous(), k, on(c["positions"]), on(c["wq"]), on(c["wk"]),
                          axis_pairs=pairs)
    assert torch.equal(y1[0], y2[0])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [2, 4])
def test_rows_off_their_alignment(io, shift):
    B, L, Hq, Hk, D, pairs = 2, 5, 3, 2, 64, (32,)
    c = case(B, L, Hq, Hk, D, pairs, io, seed=5)

    def moved(t):
        buf = torch.zeros(t.numel() + shift, dtype=t.dtype, device=DEV)
        buf[shift:] = t.reshape(-1).to(DEV)
        return buf[shift:].view(t.shape)

    run(c, pairs, io, "rms", 1e-6, "halves", q=moved(c["q"]), k=moved(c["k"]))


def test_shared_positions():
    B, L, Hq, Hk, D, pairs = 3, 5, 2, 2, 32, (8,)
    c = case(B, L, Hq, Hk, D, pairs, "fp32", seed=6)
    table = on(c["positions"])[0].contiguous()
    a = block.qk_forward(on(c["q"]), on(c["k"]), table, axis_pairs=pairs)
    b = block.qk_forward(on(c["q"]), on(c["k"]), table.expand(B, L, 1).contiguous(),
                         axis_pairs=pairs)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_zero_rows(io):
    c = case(1, 4, 3, 2, 32, (16,), io, weights=False, seed=7)
    c["q"][0, 1] = 0
    _, _, g = run(c, (16,), io, "l2", 0.0, "halves")
    assert not g["dq"][0, 1].any()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
def test_padded_batch(io, packed):
    # what lies behind a sequence's end is never read; outputs are zero there
    B, L, Hq, Hk, D, pairs = 5, 9, 3, 2, 48, (8, 8)
    lens = [9, 0, 1, 40, -3]
    eff = [9, 0, 1, 9, 0]
    c = case(B, L, Hq, Hk, D, pairs, io, seed=8)
    for b, n in enumerate(eff):
        for t in (c["q"], c["k"], *c["dy"]):
            t[b, n:] = float("nan")
    q, k = on(c["q"]), on(c["k"])
    if packed:
        q, k = block.pack8(q), block.pack8(k)
        c["q"], c["k"] = block.unpack8(q, DT[io]).cpu(), block.unpack8(k, DT[io]).cpu()
    kw = dict(norm="rms", eps=1e-6, axis_pairs=pairs)
    rest = (on(c["positions"]), on(c["wq"]), on(c["wk"]),
            torch.tensor(lens, dtype=torch.int32, device=DEV))
    y = block.qk_forward(q, k, *rest, **kw, dtype=DT[io])
    g = block.qk_backward(on(c["dy"][0]), on(c["dy"][1]), q, k, *rest, **kw)
    torch.cuda.synchronize()
    phi = phi_of(c, pairs, 1e4)
    live = np.arange(L)[None, :, None, None] < np.array(eff)[:, None, None, None]
    for i, n in enumerate("qk"):
        x, dy = (np.where(live, f64(t), 0.0) for t in (c[n], c["dy"][i]))
        w = f64(c["w" + n])
        ref, mag = bo.qk_forward(x, w, phi, "rms", 1e-6, "halves")
        close(y[i].cpu(), ref, 32 * U * mag, io)
        (dx, dw), (dxm, dwm) = bo.qk_backward(x, w, phi, "rms", 1e-6, "halves", dy)
        close(g["d" + n].cpu(), dx, 96 * U * dxm, io)
        close(g["d%s_weight" % n].cpu(), dw, (32 + B * L * 3) * U * dwm, "fp32")
        assert not y[i][~torch.from_numpy(live[..., 0, 0])].any()


# ---- 8-bit checkpoints ----

@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 4), (2, 3, 5, 16), (1, 70, 3, 112), (3, 7, 2, 72),
                                   (1, 5, 1, 256), (1, 33, 4, 20)], ids=str)
def test_pack8_bytes_are_exact(shape, io):
    rng = np.random.Generator(np.random.PCG64(9))
    x = rows(rng, shape, io)
    if x.shape[1] > 4:
        x[0, 0] = 0.0
        x[0, 1] *= 1e-30
        x[0, 2] *= 1e30
        x[0, 3, 0, 1], x[0, 3, 0, 2], x[0, 3, 0, 3] = float("inf"), float("-inf"), float("nan")
        x[0, 4, 0] = 448.0 * 2.0 ** -3        # the largest exactly at the border
    c = block.pack8(x.to(DEV))
    v, s = bo.pack8(f64(x))
    gv = c.values.view(torch.uint8).cpu().numpy()
    assert np.array_equal(c.scale.cpu().numpy(), s)
    nan = (v & 127) == 127
    assert np.array_equal(gv[~nan], v[~nan]) and np.all((gv[nan] & 127) == 127)
    for dt, out in (("bf16", torch.bfloat16), ("fp32", torch.float32)):
        back = f64(block.unpack8(c, out).cpu())
        ref = bo.unpack8(v, s)
        ok = ~np.isnan(ref)
        assert np.array_equal(np.isnan(back), ~ok)
        assert np.array_equal(back[ok], f64(torch.from_numpy(ref[ok]).to(out)))


def test_pack8_strided_and_into_slices():
    rng = np.random.Generator(np.random.PCG64(10))
    qkv = rows(rng, (2, 9, 3 * 4, 112), "bf16").to(DEV)
    x = qkv[:, :, 8:]
    c, d = block.pack8(x), block.pack8(x.contiguous())
    assert torch.equal(c.values.view(torch.uint8), d.values.view(torch.uint8))
    assert torch.equal(c.scale, d.scale)
    buf = torch.full_like(qkv, 3.0)
    block.unpack8(c, out=buf[:, :, 4:8])
    assert torch.equal(buf[:, :, 4:8], block.unpack8(c))
    assert bool((buf[:, :, :4] == 3.0).all()) and bool((buf[:, :, 8:] == 3.0).all())


def test_unpack8_takes_the_type_of_its_output():
    x = rows(np.random.Generator(np.random.PCG64(15)), (1, 5, 2, 64), "fp32").to(DEV)
    c = block.pack8(x)
    out = torch.empty_like(x)
    assert block.unpack8(c, out=out) is out
    assert torch.equal(out, block.unpack8(c, torch.float32))
    assert torch.equal(out.bfloat16(), block.unpack8(c))


def test_pack8_of_more_workgroups_than_a_grid_axis_holds():
    # 2^28 rows, 16 a workgroup, one token's repeated (pieces of two elements)
    L, H, D = (1 << 24) + 3, 16, 68
    one = rows(np.random.Generator(np.random.PCG64(16)), (H * D + 2,), "bf16").to(DEV)
    x = one[2:].view(1, 1, H, D)
    c = block.pack8(x.expand(1, L, H, D))
    ref = block.pack8(x)
    back = torch.empty(L * H * D + 2, dtype=torch.bfloat16, device=DEV)[2:].view(1, L, H, D)
    block.unpack8(c, out=back)
    want = block.unpack8(ref)
    for t in range(0, L, 1 << 21):
        part = slice(t, t + (1 << 21))
        assert bool((c.values.view(torch.uint8)[:, part] == ref.values.view(torch.uint8)).all())
        assert bool((c.scale[:, part] == ref.scale).all())
        assert bool((back[:, part] == want).all())


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[2], SHAPES[3], SHAPES[4]], ids=str)
def test_checkpoint_written_and_read(shape, pairing, io):
    pairs = shape[5]
    c = case(*shape, io, seed=11)
    kw = dict(axis_pairs=pairs, pairing=pairing)
    rest = (on(c["positions"]), on(c["wq"]), on(c["wk"]))
    q, k = on(c["q"]), on(c["k"])
    yq, yk, (cq, ck) = block.qk_forward(q, k, *rest, checkpoint=True, **kw)
    pq, pk = block.qk_forward(q, k, *rest, **kw)
    assert torch.equal(yq, pq) and torch.equal(yk, pk)
    for ckpt, x in ((cq, q), (ck, k)):
        p = block.pack8(x)
        assert torch.equal(ckpt.values.view(torch.uint8), p.values.view(torch.uint8))
        assert torch.equal(ckpt.scale, p.scale)
    # recomputation and gradients from the checkpoint: those of the rows it
    # stands for (exact in the io type)
    uq, uk = block.unpack8(cq, DT[io]), block.unpack8(ck, DT[io])
    c["q"], c["k"] = uq.cpu(), uk.cpu()
    run(c, pairs, io, "rms", 1e-6, pairing, q=uq, k=uk)
    ry = block.qk_forward(cq, ck, *rest, dtype=DT[io], **kw)
    uy = block.qk_forward(uq, uk, *rest, **kw)
    assert torch.equal(ry[0], uy[0]) and torch.equal(ry[1], uy[1])
    d = (on(c["dy"][0]), on(c["dy"][1]))
    gp = block.qk_backward(*d, cq, ck, *rest, **kw)
    gu = block.qk_backward(*d, uq, uk, *rest, **kw)
    for n in gu:
        assert torch.equal(gp[n], gu[n]), n


def test_same_bits_every_time_on_any_stream():
    shape = (2, 700, 5, 3, 112, (16, 20, 20))
    c = case(*shape, "bf16", seed=12)
    plan = block.QkPlan(*shape[:5], "bf16", DEV, axis_pairs=shape[5], weights=True,
                        checkpoint=True, backward=True)
    q, k, pos, wq, wk, d0, d1 = (on(t) for t in (c["q"], c["k"], c["positions"], c["wq"], c["wk"],
                                                 *c["dy"]))

    def once():
        y = plan.forward(q, k, pos, wq, wk)
        g = plan.backward(d0, d1, *plan.checkpoint, pos, wq, wk)
        return [t.clone() for t in (*y, *g.values())]

    first = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = once()
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_captured_and_replayed():
    shape = (1, 60, 4, 2, 112, (56,))
    c = case(*shape, "bf16", seed=13)
    plan = block.QkPlan(*shape[:5], "bf16", DEV, axis_pairs=shape[5], weights=True,
                        checkpoint=True, backward=True)
    q, k, pos, wq, wk, d0, d1 = (on(t) for t in (c["q"], c["k"], c["positions"], c["wq"], c["wk"],
                                                 *c["dy"]))

    def once():
        y = plan.forward(q, k, pos, wq, wk)
        return list(y) + list(plan.backward(d0, d1, *plan.checkpoint, pos, wq, wk).values())

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = once()
    for i in range(4):
        q.mul_(1.25)
        d1.add_(0.5 * i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = once()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_backward_into_given_gradients_makes_none_of_its_own():
    shape = (1, 40, 3, 2, 64, (32,))
    c = case(*shape, "bf16", seed=17)
    q, k, pos, wq, wk, d0, d1 = (on(t) for t in (c["q"], c["k"], c["positions"], c["wq"], c["wk"],
                                                 *c["dy"]))
    plan = block.QkPlan(*shape[:5], "bf16", DEV, axis_pairs=shape[5], weights=True)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    g = plan.backward(d0, d1, q, k, pos, wq, wk, dq=dq, dk=dk)
    assert g["dq"] is dq and g["dk"] is dk and plan.dq is None and plan.dk is None
    got = [t.clone() for t in g.values()]
    for a, b in zip(got, plan.backward(d0, d1, q, k, pos, wq, wk, dk=dk).values()):
        assert torch.equal(a, b)
    assert plan.dk is None and plan.dq is not None
