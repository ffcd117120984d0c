"""The block's operators together, as a training step of one block uses them:
the recurrence over the projection's rows, queries and keys normalised and
rotated out of them, the mixer, and the way back from the 8-bit checkpoints
with q', k' formed again; against the float64 oracles run on the values that
each operator was handed."""

import numpy as np
import pytest
import torch

import oracle
from gated_deltanet_recurrence_frame_amd import binding as gb
from gated_deltanet_recurrence_frame_amd import block
from gated_deltanet_recurrence_frame_amd import inputs as gin
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def f64(t):
    return gin.as_f64(t.cpu())


def rel(a, b):
    a = f64(a)
    assert np.isfinite(a).all()
    return np.linalg.norm((a - b).ravel()) / np.linalg.norm(b.ravel())


@pytest.mark.parametrize("io,tol", [("bf16", 2e-2), ("fp32", 1e-5)])
def test_training_step_of_a_block(io, tol):
    # the bars of the mixer's own parity tests; checkpoints are exact values
    # to the operators that read them, so they add nothing
    B, T, N, H, D, pairs = 1, 6, 40, 4, 112, (16, 20, 20)
    L, C = T * N, H * D
    rng = np.random.Generator(np.random.PCG64(21))
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    qkvz = torch.from_numpy(rng.standard_normal((B, L, 4 * C))).to(dt)
    qkvz[..., 3 * C:] += 2.0
    qkvz = qkvz.to(DEV)
    pos = torch.from_numpy(np.stack([np.arange(L) // N, np.arange(L) % N // 8,
                                     np.arange(L) % 8], -1)[None]).to(torch.int32).to(DEV)
    w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).float().to(DEV) for _ in range(2)]
    gamma = torch.from_numpy(rng.uniform(0.9, 1, (B, T, H))).float().to(DEV)
    beta = torch.from_numpy(rng.uniform(0, 1, (B, L, H))).float().to(DEV)
    d_o = torch.from_numpy(rng.standard_normal((B, L, H, D))).to(dt).to(DEV)
    heads = qkvz.view(B, L, 4 * H, D)
    q, k = heads[:, :, :H], heads[:, :, H:2 * H]

    # forward: v is the recurrence's output over its projected rows
    rec = block.LrecPlan(B, L, C, io, DEV, True, True, saved=True, backward=True)
    v, _ = rec.forward(qkvz[..., 2 * C:3 * C], qkvz[..., 3 * C:])
    v = v.view(B, L, H, D)
    qk = block.QkPlan(B, L, H, H, D, io, DEV, norm="rms", axis_pairs=pairs, weights=True,
                      checkpoint=True, backward=True)
    q1, k1 = qk.forward(q, k, pos, *w)
    o, state, saved = gb.forward(q1, k1, v, gamma, beta, N, return_saved=True)
    ref_v, _ = bo.lrec_forward(f64(qkvz[..., 2 * C:3 * C]), f64(qkvz[..., 3 * C:]), True, True)
    assert rel(v.reshape(B, L, C), ref_v[0]) <= tol
    ro, rs = oracle.forward(f64(q1), f64(k1), f64(v), f64(gamma), f64(beta), N)
    assert rel(o, ro) <= tol and rel(state, rs) <= tol

    # backward from the checkpoints: v and q', k' formed again, the mixer's
    # gradients, then the two operators' into one projection gradient
    cv = block.pack8(v)
    v8 = block.unpack8(cv, dt)
    again = block.QkPlan(B, L, H, H, D, io, DEV, norm="rms", axis_pairs=pairs)
    q8, k8 = again.forward(*qk.checkpoint, pos, *w)
    g = gb.backward(q8, k8, v8, gamma, beta, N, d_o)
    rg = oracle.backward(f64(q8), f64(k8), f64(v8), f64(gamma), f64(beta), N, f64(d_o))
    for n in ("dq", "dk", "dv"):
        assert rel(g[n], rg[n]) <= tol, n
    d = torch.zeros_like(qkvz)
    dh = d.view(B, L, 4 * H, D)
    out = qk.backward(g["dq"], g["dk"], *qk.checkpoint, pos, *w, dq=dh[:, :, :H],
                      dk=dh[:, :, H:2 * H])
    rec.backward(qkvz[..., 2 * C:3 * C], qkvz[..., 3 * C:], g["dv"].view(B, L, C),
                 saved=rec.saved, dx=d[..., 2 * C:3 * C], dgate=d[..., 3 * C:])
    torch.cuda.synchronize()
    phi = bo.qk_angles(f64(pos), pairs, 1e4)
    for i, n in enumerate("qk"):
        c = qk.checkpoint[i]
        x = bo.unpack8(c.values.view(torch.uint8).cpu().numpy(), c.scale.cpu().numpy())
        (dx, dw), _ = bo.qk_backward(x, f64(w[i]), phi, "rms", 1e-6, "halves", f64(g["d" + n]))
        assert rel(dh[:, :, i * H:(i + 1) * H], dx) <= tol
        assert rel(out["d%s_weight" % n], dw) <= tol
        # the checkpoint's own error: at most half a step of e4m3
        assert rel(block.unpack8(c, torch.float32), f64((q, k)[i])) <= 2.0 ** -4
    (dx, dz, _), _ = bo.lrec_backward(f64(qkvz[..., 2 * C:3 * C]), f64(qkvz[..., 3 * C:]), True,
                                      True, f64(g["dv"].reshape(B, L, C)))
    assert rel(d[..., 2 * C:3 * C], dx) <= tol and rel(d[..., 3 * C:], dz) <= tol
    # gradients through the checkpoints stay near those of the exact rows
    exact = gb.backward(q1, k1, v, gamma, beta, N, d_o, saved=saved)
    for n in ("dq", "dk", "dv"):
        assert rel(g[n], f64(exact[n])) <= 0.2, n


def test_streaming_step_by_step():
    # frame by frame: the prologue at the frame's positions, then gdn_step;
    # equal to the whole clip at once within the mixer's bar
    B, T, N, H, D, pairs = 1, 4, 24, 4, 64, (8, 12, 12)
    L = T * N
    rng = np.random.Generator(np.random.PCG64(22))
    qk, v = (torch.from_numpy(rng.standard_normal((B, L, h, D))).bfloat16().to(DEV)
             for h in (2 * H, H))
    pos = torch.from_numpy(np.stack([np.arange(L) // N, np.arange(L) % N // 6,
                                     np.arange(L) % 6], -1)[None]).to(torch.int32).to(DEV)
    gamma = torch.from_numpy(rng.uniform(0.9, 1, (B, T, H))).float().to(DEV)
    beta = torch.from_numpy(rng.uniform(0, 1, (B, L, H))).float().to(DEV)
    kw = dict(norm="l2", eps=0.0, axis_pairs=pairs)
    q1, k1 = block.qk_forward(qk[:, :, :H], qk[:, :, H:], pos, **kw)
    ro, rs = oracle.forward(f64(q1), f64(k1), f64(v), f64(gamma), f64(beta), N)
    plan = block.QkPlan(B, N, H, H, D, "bf16", DEV, **kw)
    step = gb.StepPlan(B, H, N, D, "bf16", DEV)
    state, outs = torch.zeros((B, H, D, D), device=DEV), []
    for t in range(T):
        s = slice(t * N, (t + 1) * N)
        qf, kf = plan.forward(qk[:, s, :H], qk[:, s, H:], pos[:, s].contiguous())
        assert torch.equal(qf, q1[:, s]) and torch.equal(kf, k1[:, s])
        outs.append(step(qf, kf, v[:, s].contiguous(), gamma[:, t:t + 1].contiguous(),
                         beta[:, s].contiguous(), state).clone())
    assert rel(torch.cat(outs, 1), ro) <= 2e-2 and rel(state, rs) <= 2e-2
