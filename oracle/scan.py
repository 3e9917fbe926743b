"""fp64 oracle of the elementwise gated linear recurrence and its 8-bit checkpoint -- TEST INFRASTRUCTURE.

    h_t = alpha_t h_{t-1} + w_t x_t,   alpha_t = exp(lambda_t),   w_t = 1 or 1 - alpha_t

Token by token in numpy, sequence by sequence; shares nothing with the CUDA
library.  Pinned in tests/test_oracle_scan.py by closed forms, by central
differences and by torch autograd through a plain loop.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, np.float64)


def log_gate(g, raw):
    """lambda of the gates g: g itself, or log sigmoid(g)."""
    g = _f64(g)
    return np.minimum(g, 0.0) - np.log1p(np.exp(-np.abs(g))) if raw else g


def spans(B, T, cu=None):
    """(row of states, b, first row, one past the last row) of every sequence."""
    if cu is None:
        return [(b, b, 0, T) for b in range(B)]
    cu = [int(v) for v in cu]
    return [(i, 0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def _states(s, n, D):
    return np.zeros((n, D)) if s is None else _f64(s)


def forward(x, g, s0=None, *, raw=False, complement=False, cu=None):
    """(h, final state, z): z_t = h_{t-1}, less x_t with ``complement``: what the checkpoint keeps beside
    lambda.  Rows outside every sequence are zero."""
    x, lam = _f64(x), log_gate(g, raw)
    B, T, D = x.shape
    seqs = spans(B, T, cu)
    s0 = _states(s0, len(seqs), D)
    h, z, sT = np.zeros_like(x), np.zeros_like(x), s0.copy()
    with np.errstate(all="ignore"):
        alpha = np.exp(lam)
        u = -np.expm1(lam) * x if complement else x
        for i, b, lo, hi in seqs:
            c = s0[i]
            for t in range(lo, hi):
                z[b, t] = c - x[b, t] if complement else c
                c = alpha[b, t] * c + u[b, t]
                h[b, t] = c
            sT[i] = c
    return h, sT, z


def saved(x, h, s0=None, *, complement=False, cu=None):
    """z from the forward's output h as it was stored."""
    x, h = _f64(x), _f64(h)
    B, T, D = h.shape
    seqs = spans(B, T, cu)
    s0 = _states(s0, len(seqs), D)
    z = np.zeros_like(h)
    for i, b, lo, hi in seqs:
        if hi > lo:
            z[b, lo] = s0[i]
            z[b, lo + 1:hi] = h[b, lo:hi - 1]
            if complement:
                z[b, lo:hi] -= x[b, lo:hi]
    return z


def backward(lam, z, dh, dsT=None, *, raw=False, complement=False, cu=None):
    """dict dx, dg, dS0 and d (dL/dh_t with what later rows pass back) of the recurrence with log-gates lam
    and z as above; dg is with respect to the raw gate with ``raw``."""
    lam, z, dh = _f64(lam), _f64(z), _f64(dh)
    B, T, D = dh.shape
    seqs = spans(B, T, cu)
    dsT = _states(dsT, len(seqs), D)
    d, ds0 = np.zeros_like(dh), dsT.copy()
    with np.errstate(all="ignore"):
        alpha, beta = np.exp(lam), -np.expm1(lam)
        for i, b, lo, hi in seqs:
            c = dsT[i]
            for t in range(hi - 1, lo - 1, -1):
                d[b, t] = dh[b, t] + c
                c = alpha[b, t] * d[b, t]
            ds0[i] = c
        dg = alpha * d * z
        out = dict(dx=beta * d if complement else d.copy(), dg=dg * beta if raw else dg, dS0=ds0, d=d)
        for b, t in _outside(B, T, seqs):
            out["dx"][b, t] = out["dg"][b, t] = 0.0
    return out


def _outside(B, T, seqs):
    own = np.zeros((B, T), bool)
    for _, b, lo, hi in seqs:
        own[b, lo:hi] = True
    return [tuple(p) for p in np.argwhere(~own)]


def scan_abs(alpha, u, first, reverse=False):
    """E_t = alpha_t E_{t-1} + S_t with S_t = alpha_t S_{t-1} + |u_t|, rows where ``first`` [B, T] start anew
    (``reverse``: from the last row on, alpha_t then the factor into row t): the sum of the magnitudes of
    h_t's terms, each as often as the roundings it has passed."""
    alpha, u = np.abs(alpha), np.abs(u)
    S, E = np.zeros_like(u), np.zeros_like(u)
    B, T, _ = u.shape
    step = range(T - 1, -1, -1) if reverse else range(T)
    prev = 1 if reverse else -1
    for t in step:
        for b in range(B):
            if first[b, t] or not 0 <= t + prev < T:
                S[b, t] = u[b, t]
                E[b, t] = S[b, t]
            else:
                S[b, t] = alpha[b, t] * S[b, t + prev] + u[b, t]
                E[b, t] = alpha[b, t] * E[b, t + prev] + S[b, t]
    return S, E


# ----------------------------------------------------------------- checkpoint
LEAST = -128.0  # lambda is held no lower: exp of it is zero in fp32


def layout(rows, D):
    """(P, K, byte offsets of lambda codes, z codes, lambda scales, z scales, and the size)."""
    up = lambda v: -(-v // 256) * 256
    P, K = -(-D // 16) * 16, -(-D // BLOCK)
    codes, scales = up(rows * P), up(rows * K)
    return P, K, (0, codes, 2 * codes, 2 * codes + scales, 2 * (codes + scales))


def scale_exponent(v):
    """k of one block's values: the least integer >= -126 with max |v| <= 448 * 2^k over the finite values."""
    v = np.abs(np.asarray(v, np.float64))
    top = np.max(np.where(np.isfinite(v), v, 0.0), axis=-1)
    m, e = np.frexp(np.where(top > 0, top, 1.0))         # top = m 2^e, 1/2 <= m < 1;  448 = 7/8 * 2^9
    return np.where(top > 0, np.maximum(e - 9 + (m > 0.875), -126), -126)


def round_e4m3(q):
    """q (|q| <= 448) to 4 significant bits, no finer than 2^-9, to nearest even."""
    q = np.asarray(q, np.float64)
    _, e = np.frexp(np.where(q == 0, 1.0, np.where(np.isfinite(q), q, 1.0)))
    step = np.exp2(np.maximum(e - 1, -6) - 3)
    return np.where(np.isfinite(q), np.rint(q / step) * step, np.nan)


def quantise(v):
    """(values as the checkpoint holds them, scales 2^k [..., K]) of v [..., D]."""
    v = _f64(v)
    D, K = v.shape[-1], -(-v.shape[-1] // BLOCK)
    out, scale = np.empty_like(v), np.empty(v.shape[:-1] + (K,))
    for j in range(K):
        s = slice(j * BLOCK, min(D, (j + 1) * BLOCK))
        scale[..., j] = np.exp2(scale_exponent(v[..., s]).astype(np.float64))
        out[..., s] = round_e4m3(v[..., s] / scale[..., j:j + 1]) * scale[..., j:j + 1]
    return out, scale


def unpack(buf, B, T, D):
    """(lambda, z, lambda scales [B, T, K], z scales) of a checkpoint's bytes (numpy uint8)."""
    rows = B * T
    P, K, at = layout(rows, D)
    out, scales = [], []
    for i in range(2):
        c = buf[at[i]:at[i] + rows * P].reshape(rows, P)[:, :D].astype(np.int64)
        e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
        v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))
        v = np.where((c & 127) == 127, np.nan, np.where(c >= 128, -v, v))
        s = np.exp2(buf[at[2 + i]:at[2 + i] + rows * K].reshape(K, rows).T.astype(np.float64) - 127)
        out.append((v * np.repeat(s, BLOCK, axis=1)[:, :D]).reshape(B, T, D))
        scales.append(s.reshape(B, T, K))
    return out[0], out[1], scales[0], scales[1]
