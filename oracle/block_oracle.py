"""Float64 CPU oracle of the block's operators (gdn_block.h).

TEST INFRASTRUCTURE ONLY, like ``gdn_oracle``: it shares no code with the
library.  Besides every result it gives a *magnitude*: the same formula with
every product and sum of absolute values, which is what rounding errors of a
32-bit evaluation are proportional to.  The tests derive their element-wise
tolerances from it.

Pinned by ``tests/test_block_oracle.py`` (closed forms, brute force, finite
differences).
"""

import numpy as np

__all__ = ["qk_angles", "qk_forward", "qk_backward", "pack8", "unpack8", "e4m3_values",
           "lrec_forward", "lrec_backward"]


# ---- queries and keys ---------------------------------------------------

def qk_angles(positions, axis_pairs, theta):
    """phi [B, L, P] of positions [B, L, axes]: pair f of axis a's n_a pairs
    turns by positions[..., a] * theta ** (-f / n_a)."""
    cols = []
    for a, n in enumerate(axis_pairs):
        f = np.arange(n, dtype=np.float64)
        cols.append(np.asarray(positions, dtype=np.float64)[..., a:a + 1] * theta ** (-f / n))
    return np.concatenate(cols, axis=-1)


def _pair_index(P, pairing):
    m = np.arange(P)
    return (m, m + P) if pairing == "halves" else (2 * m, 2 * m + 1)


def _turn(x, phi, pairing, sign):
    """Rows x [B, L, H, D] with their pairs turned by sign * phi, and the
    magnitude |x_i| + |x_j| of each turned element."""
    y, mag = x.copy(), np.abs(x)
    if phi is None or phi.shape[-1] == 0:
        return y, mag
    i, j = _pair_index(phi.shape[-1], pairing)
    c, s = np.cos(phi)[:, :, None], sign * np.sin(phi)[:, :, None]
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    both = np.abs(x[..., i]) + np.abs(x[..., j])
    mag[..., i] = both
    mag[..., j] = both
    return y, mag


def _inverse(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    ss = np.sum(x * x, axis=-1, keepdims=True)
    ss = (ss / x.shape[-1] if norm == "rms" else ss) + eps
    with np.errstate(divide="ignore"):
        return np.where(ss > 0, 1.0 / np.sqrt(ss), 0.0)


def qk_forward(x, w, phi, norm, eps, pairing):
    """(y, magnitude) for one operand x [B, L, H, D]; w [D] or None; phi
    [B, L, P] or None."""
    x = np.asarray(x, dtype=np.float64)
    n = x * _inverse(x, norm, eps)
    if w is not None:
        n = n * np.asarray(w, dtype=np.float64)
    return _turn(n, phi, pairing, 1.0)


def qk_backward(x, w, phi, norm, eps, pairing, dy):
    """dx, dw (None without a norm) and their magnitudes."""
    dy = np.asarray(dy, dtype=np.float64)
    g, gm = _turn(dy, phi, pairing, -1.0)
    if norm == "none":
        return (g, None), (gm, None)
    x = np.asarray(x, dtype=np.float64)
    r = _inverse(x, norm, eps)
    xr = x * r
    dw, dwm = np.sum(g * xr, axis=(0, 1, 2)), np.sum(gm * np.abs(xr), axis=(0, 1, 2))
    wv = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    g, gm = g * wv, gm * np.abs(wv)
    c = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    dx = r * (g - xr * (c * np.sum(xr * g, axis=-1, keepdims=True)))
    dxm = r * (gm + np.abs(xr) * (c * np.sum(np.abs(xr) * gm, axis=-1, keepdims=True)))
    return (dx, dw), (dxm, dwm)


# ---- 8-bit checkpoints --------------------------------------------------

def e4m3_values():
    """The 256 values of OCP e4m3 (bias 7, no infinity, 0x7f and 0xff NaN),
    from the format's definition."""
    out = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            v = np.nan
        elif e == 0:
            v = m * 2.0 ** -9
        else:
            v = (1.0 + m / 8.0) * 2.0 ** (e - 7)
        out[b] = -v if s else v
    return out


def pack8(x):
    """(bytes, scale bytes) of rows x [..., D]: the nearest of the format's
    values by search, ties to the even byte."""
    x = np.asarray(x, dtype=np.float64)
    rows = x.reshape(-1, x.shape[-1])
    grid = e4m3_values()[:127]           # 0 .. 448, ascending with the byte
    v = np.empty(rows.shape, dtype=np.uint8)
    scale = np.empty(rows.shape[0], dtype=np.uint8)
    for i, row in enumerate(rows):
        fin = np.abs(row[np.isfinite(row)])
        amax = fin.max() if fin.size else 0.0
        s = 0
        while amax > 448.0 * 2.0 ** (s - 127):
            s += 1
        scale[i] = s
        a = np.abs(row) * 2.0 ** (127.0 - s)
        ok = np.isfinite(row)
        a = np.where(ok, a, 0.0)
        hi = np.clip(np.searchsorted(grid, a, side="left"), 1, 126)
        lo = hi - 1
        dl, dh = a - grid[lo], grid[hi] - a
        up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
        b = np.where(up, hi, lo)
        b = np.where(ok, b, 127)
        v[i] = np.where(np.signbit(row) & ok, b | 128, b)
    return v.reshape(x.shape), scale.reshape(x.shape[:-1])


def unpack8(v, scale):
    return e4m3_values()[np.asarray(v)] * 2.0 ** (np.asarray(scale, dtype=np.float64) - 127.0)[
        ..., None]


# ---- gated linear recurrence --------------------------------------------

_U = 2.0 ** -24
# A 32-bit sigmoid below the smallest normal number may be flushed to zero
# (the hardware's exp2 does): at |z| > 87.3, an absolute error of up to 2^-126
# in a or 1 - a, whatever they multiply.
_TINY = 2.0 ** -126


def _gates(z, logits):
    z = np.asarray(z, dtype=np.float64)
    if not logits:
        return z, 1.0 - z, np.zeros_like(z)
    with np.errstate(over="ignore"):
        # (relative error of a 32-bit sigmoid grows with |z| where it is small)
        return 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z)), np.abs(np.where(
            np.isfinite(z), z, 0.0))


def lrec_forward(x, z, logits, complement, h0=None, lengths=None):
    """o [B, L, C], final state [B, C], and bounds of a 32-bit evaluation's
    errors in them.

    The bound: a contribution u_s to h_t is multiplied by t - s gates, each
    product with the gate's own relative error (at most 8 roundings and, for a
    logit, |z| more) and a rounding or two of the sum it enters; the chunked
    evaluation regroups the same products.  So with m_t = |a_t| m_{t-1} + |u_t|
    and k_t = (12 + |z_t|) 2^-24,
      e_t = |a_t| (e_{t-1} + k_t m_{t-1}) + k_t |u_t|,
    and 2^-126 (m_{t-1} + |x_t|) for gates that are flushed to zero."""
    x = np.asarray(x, dtype=np.float64)
    B, L, C = x.shape
    a, na, za = _gates(z, logits)
    k = (12.0 + za) * _U
    u = na * x if complement else x
    h = np.zeros((B, C)) if h0 is None else np.array(h0, dtype=np.float64)
    m, e = np.abs(h), np.zeros((B, C))
    o, eo = np.zeros((B, L, C)), np.zeros((B, L, C))
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)
    for t in range(L):
        on = (t < n)[:, None]
        ab, ub = np.abs(a[:, t]), np.abs(u[:, t])
        e = np.where(on, ab * (e + k[:, t] * m) + k[:, t] * ub +
                     _TINY * (m + np.abs(x[:, t])), e)
        m = np.where(on, ab * m + ub, m)
        h = np.where(on, a[:, t] * h + u[:, t], h)
        o[:, t] = np.where(on, h, 0.0)
        eo[:, t] = np.where(on, e, 0.0)
    return (o, h), (eo, e)


def lrec_backward(x, z, logits, complement, d_o, h0=None, dhT=None, lengths=None):
    """dx, dz, dh0 and bounds of a 32-bit evaluation's errors (lrec_forward's
    recursion, run from the end for G, and first-order products of both)."""
    x = np.asarray(x, dtype=np.float64)
    d_o = np.asarray(d_o, dtype=np.float64)
    B, L, C = x.shape
    a, na, za = _gates(z, logits)
    k = (12.0 + za) * _U
    u = na * x if complement else x
    h = np.zeros((B, C)) if h0 is None else np.array(h0, dtype=np.float64)
    m, e = np.abs(h), np.zeros((B, C))
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)
    prev, pm, pe = (np.zeros((B, L, C)) for _ in range(3))
    for t in range(L):
        prev[:, t], pm[:, t], pe[:, t] = h, m, e
        on = (t < n)[:, None]
        ab, ub = np.abs(a[:, t]), np.abs(u[:, t])
        e = np.where(on, ab * (e + k[:, t] * m) + k[:, t] * ub +
                     _TINY * (m + np.abs(x[:, t])), e)
        m = np.where(on, ab * m + ub, m)
        h = np.where(on, a[:, t] * h + u[:, t], h)
    c = np.zeros((B, C)) if dhT is None else np.array(dhT, dtype=np.float64)
    cm, ce = np.abs(c), np.zeros((B, C))
    dx, dz, ex, ez = (np.zeros((B, L, C)) for _ in range(4))
    for t in range(L - 1, -1, -1):
        on = (t < n)[:, None]
        kt = k[:, t]
        G = d_o[:, t] + c
        Gm = np.abs(d_o[:, t]) + cm
        Ge = ce + 2.0 * _U * Gm
        f = prev[:, t] - (x[:, t] if complement else 0.0)
        fm = pm[:, t] + (np.abs(x[:, t]) if complement else 0.0)
        fe = pe[:, t] + 2.0 * _U * fm
        s = np.abs(a[:, t] * na[:, t]) if logits else 1.0
        v = G * f * (a[:, t] * na[:, t] if logits else 1.0)
        dz[:, t] = np.where(on, v, 0.0)
        ez[:, t] = np.where(on, s * (Ge * fm + Gm * fe + 4.0 * kt * Gm * fm) + _TINY * Gm * fm,
                            0.0)
        w = np.abs(na[:, t]) if complement else 1.0
        dx[:, t] = np.where(on, G * (na[:, t] if complement else 1.0), 0.0)
        ex[:, t] = np.where(on, w * (Ge + 2.0 * kt * Gm) + _TINY * Gm, 0.0)
        ab = np.abs(a[:, t])
        ce = np.where(on, ab * (Ge + kt * Gm) + _TINY * Gm, ce)
        cm = np.where(on, ab * Gm, cm)
        c = np.where(on, a[:, t] * G, c)
    return (dx, dz, c), (ex, ez, ce)
