"""fp64 reference of the selective state-space mixer (plain numpy, token by token; no code shared with the
GPU path): prologue, scan, decode step, block norm, and their gradients from the same recurrences walked
backwards.

    H_t = e^{g_t} H_{t-1} + step_t B_t x_t^T,   y_t = H_t^T C_t + d x_t      (per head; B, C per group)
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def softplus(v):
    return np.logaddexp(0.0, v)


def spans(B, T, offsets):
    """[(first row, row past the last)] of every sequence in flattened rows."""
    if offsets is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return [(int(offsets[b]), int(offsets[b + 1])) for b in range(len(offsets) - 1)]


# ---- prologue -------------------------------------------------------------------------------------------

def prologue(xbc, delta, w, bias, a, delta_bias, seqs, state=None, silu=True):
    """xbc [rows, ch], delta [rows, H], seqs from spans(); state [B, 3, ch]. Returns u, step, g, new state."""
    v = np.zeros_like(xbc)
    new = None if state is None else state.copy()
    for b, (lo, hi) in enumerate(seqs):
        full = np.concatenate([np.zeros((3, xbc.shape[1])) if state is None else state[b], xbc[lo:hi]])
        for j in range(4):
            v[lo:hi] += w[:, j] * full[j:j + hi - lo]
        v[lo:hi] += 0.0 if bias is None else bias
        if state is not None:
            new[b] = full[-3:]
    step = softplus(delta + delta_bias)
    return (v * sigmoid(v) if silu else v), step, a * step, new


def prologue_grad(xbc, delta, w, bias, a, delta_bias, du, dstep, dg, seqs, silu=True):
    """Returns dxbc, ddelta, dw, dbias, da, ddelta_bias (zero initial states)."""
    v, _, _, _ = prologue(xbc, delta, w, bias, a, delta_bias, seqs, silu=False)
    s = sigmoid(v)
    dv = du * (s * (1 + v * (1 - s)) if silu else 1.0)
    dx, dw = np.zeros_like(xbc), np.zeros_like(w)
    for lo, hi in seqs:
        for t in range(lo, hi):
            for j in range(4):
                if t - 3 + j >= lo:
                    dx[t - 3 + j] += w[:, j] * dv[t]
                    dw[:, j] += dv[t] * xbc[t - 3 + j]
    z = delta + delta_bias
    dz = (dstep + a * dg) * sigmoid(z)
    return dx, dz, dw, dv.sum(0), (dg * softplus(z)).sum(0), dz.sum(0)


# ---- scan -----------------------------------------------------------------------------------------------

def scan(x, step, g, bm, cm, d, s0, seqs):
    """x [rows, H, P], step, g [rows, H], bm, cm [rows, G, N], d [H] or None, s0 [B, H, N, P] or None.
    Returns y [rows, H, P] and the final states."""
    rows, H, P = x.shape
    G, N = bm.shape[1:]
    of = np.arange(H) // (H // G)
    y = np.zeros_like(x)
    s1 = np.zeros((len(seqs), H, N, P)) if s0 is None else np.array(s0, dtype=np.float64)
    for b, (lo, hi) in enumerate(seqs):
        h = s1[b]
        for t in range(lo, hi):
            h = np.exp(g[t])[:, None, None] * h + bm[t][of][:, :, None] * (step[t][:, None] * x[t])[:, None, :]
            y[t] = np.einsum("hn,hnp->hp", cm[t][of], h)
        s1[b] = h
    return y + (0.0 if d is None else d[:, None] * x), s1


def scan_grad(x, step, g, bm, cm, d, s0, seqs, dy, ds1=None):
    """Returns dx, dstep, dg, dbm, dcm, dd, ds0: H_t kept for every token, adjoint walked backwards."""
    rows, H, P = x.shape
    G, N = bm.shape[1:]
    of = np.arange(H) // (H // G)
    dx, dstep, dg, dbm, dcm = (np.zeros_like(t) for t in (x, step, g, bm, cm))
    ds0 = np.zeros((len(seqs), H, N, P)) if ds1 is None else np.array(ds1, dtype=np.float64)
    dsk = np.zeros(H) if d is None else d
    for b, (lo, hi) in enumerate(seqs):
        hs = [np.zeros((H, N, P)) if s0 is None else np.asarray(s0[b], dtype=np.float64)]
        for t in range(lo, hi):
            hs.append(np.exp(g[t])[:, None, None] * hs[-1] + bm[t][of][:, :, None] * (step[t][:, None] * x[t])[:, None, :])
        dh = ds0[b]
        for t in range(hi - 1, lo - 1, -1):
            dh = dh + cm[t][of][:, :, None] * dy[t][:, None, :]
            u = np.einsum("hn,hnp->hp", bm[t][of], dh)
            dx[t] = step[t][:, None] * u + dsk[:, None] * dy[t]
            dstep[t] = (x[t] * u).sum(-1)
            np.add.at(dcm[t], of, np.einsum("hnp,hp->hn", hs[t - lo + 1], dy[t]))
            np.add.at(dbm[t], of, step[t][:, None] * np.einsum("hnp,hp->hn", dh, x[t]))
            dh = np.exp(g[t])[:, None, None] * dh
            dg[t] = (dh * hs[t - lo]).sum((1, 2))
        ds0[b] = dh
    return dx, dstep, dg, dbm, dcm, (x * dy).sum((0, 2)), ds0


def decode(xbc, delta, w, bias, a, delta_bias, d, conv_state, state):
    """One token per row: xbc [B, ch], delta [B, H], conv_state [B, 3, ch], state [B, H, N, P]. Returns y and
    the new states."""
    B, H, N, P = state.shape
    G = (xbc.shape[1] - H * P) // (2 * N)
    seqs = [(b, b + 1) for b in range(B)]
    u, step, g, conv = prologue(xbc, delta, w, bias, a, delta_bias, seqs, conv_state)
    x, bm, cm = u[:, :H * P].reshape(B, H, P), u[:, H * P:H * P + G * N].reshape(B, G, N), u[:, H * P + G * N:].reshape(B, G, N)
    y, s1 = scan(x, step, g, bm, cm, d, state, seqs)
    return y, conv, s1


# ---- block norm -----------------------------------------------------------------------------------------

def _parts(x, z, post, residual, scale, pre, groups, eps):
    t = x if z is None else x * z * sigmoid(z)
    tg = t.reshape(t.shape[0], groups, -1)
    inv_t = 1 / np.sqrt((tg ** 2).mean(-1, keepdims=True) + eps)
    th = (tg * inv_t).reshape(t.shape)
    p = t if post is None else th * post
    r = (0.0 if residual is None else residual) + (p if scale is None else p * scale)
    inv_r = 1 / np.sqrt((r ** 2).mean(-1, keepdims=True) + eps)
    return th, inv_t, p, r, inv_r


def block_norm(x, z, post, residual, scale, pre, groups=1, eps=1e-5):
    """Returns r and n (None without pre)."""
    *_, r, inv_r = _parts(x, z, post, residual, scale, pre, groups, eps)
    return r, None if pre is None else r * inv_r * pre


def block_norm_grad(x, z, post, residual, scale, pre, d_r, d_n, groups=1, eps=1e-5):
    """Returns dx, dz, dpost, dresidual, dscale, dpre."""
    th, inv_t, p, r, inv_r = _parts(x, z, post, residual, scale, pre, groups, eps)
    dr = np.zeros_like(r) if d_r is None else d_r.copy()
    dpre = dz = dpost = None
    if pre is not None:
        nh = r * inv_r
        dpre = (d_n * nh).sum(0)
        k = d_n * pre
        dr += inv_r * (k - nh * (k * nh).mean(-1, keepdims=True))
    dp = dr if scale is None else dr * scale
    dt = dp
    if post is not None:
        dpost = (dp * th).sum(0)
        k, tg = (dp * post).reshape(len(x), groups, -1), th.reshape(len(x), groups, -1)
        dt = (inv_t * (k - tg * (k * tg).mean(-1, keepdims=True))).reshape(x.shape)
    dx = dt
    if z is not None:
        s = sigmoid(z)
        dx, dz = dt * z * s, dt * x * s * (1 + z * (1 - s))
    return dx, dz, dpost, dr, None if scale is None else (dr * p).sum(0), dpre
