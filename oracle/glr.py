"""fp64 gated linear recurrence with a vector state, written from its formulas
(include/gdn_glr.h), token by token, with bounds of an fp32 evaluation.

    h_t = a_t h_{t-1} + b_t,  a = exp(g),  b = x or (1 - a) x

and its reverse mode.  No chunks: the chunk schedule of the CUDA kernels is a
reordering of this computation.  Arrays are numpy; shapes as in the header.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32


def _parts(x, g, complement):
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    a = np.exp(g)
    gain = -np.expm1(g) if complement else np.ones_like(g)
    return x, a, gain


def forward(x, g, lengths, h0=None, complement=False):
    """Returns (h [T, D], s_final [N, D])."""
    x, a, gain = _parts(x, g, complement)
    h = np.zeros_like(x)
    s = np.zeros((len(lengths), x.shape[1])) if h0 is None else np.array(h0, np.float64)
    t = 0
    for n, L in enumerate(lengths):
        for _ in range(L):
            s[n] = a[t] * s[n] + gain[t] * x[t]
            h[t] = s[n]
            t += 1
    return h, s


def backward(x, g, lengths, d_h, h0=None, ds_final=None, complement=False):
    """Returns (dx, dg [T, D], dh0 [N, D])."""
    h, _ = forward(x, g, lengths, h0, complement)
    x, a, gain = _parts(x, g, complement)
    d_h = np.asarray(d_h, np.float64)
    N, D = len(lengths), x.shape[1]
    dx, dg = np.zeros_like(x), np.zeros_like(x)
    u = np.zeros((N, D)) if ds_final is None else np.array(ds_final, np.float64)
    start = 0
    for n, L in enumerate(lengths):
        for t in range(start + L - 1, start - 1, -1):
            first = t == start
            before = h[t - 1] if not first else (0.0 if h0 is None else np.asarray(h0[n], np.float64))
            lam = d_h[t] + u[n]
            u[n] = a[t] * lam
            dx[t] = gain[t] * lam
            dg[t] = u[n] * (before - x[t] if complement else before)
        start += L
    return dx, dg, u


# One step of an fp32 evaluation multiplies every older term by a decay that is
# off by
#   |g| < 1/8, plain: the series 1 + g s, whose rest is 0.1 U of a and whose s is
#     off by 1.1 U (half a step of s, which may be above 1, and |g| times the step
#     before), that is 0.14 U of a, and half a step of a (U above 1): 1.4 U
#   |g| < 1/2, complement: e = exp(g) - 1 is off by 2.9 U of itself (s by 1.7 U, its
#     product with g by U, the rest 0.25 U), at most 1.9 U of a = 1 + e, whose
#     rounding is at most 0.83 U below 1 and U above: 2.9 U
#   else (4 + 1.25 |g|) U: 2^x off by 4 U, the rounding of x = g log2 e by |g| U and
#     that of the constant by |g| U / 4
# and adds one rounding of the running product and one of the running sum: 2 U.
# A term starts with the rounding of its input ((1 - a) x: at most 14 U) and ends
# with those of the state's last operations: 16 U.  First order; the factor 1.01
# covers the products of roundings at these lengths.
ENDS = 16.0 * 1.01 * U


def decay_bound(g, complement=False):
    """Bound of an fp32 decay's relative error."""
    size = np.abs(np.asarray(g, np.float64))
    near, most = (0.5, 2.9) if complement else (0.125, 1.4)
    return U * np.where(size < near, most, 4.0 + 1.25 * np.minimum(size, 200.0))


def _step(g, complement):
    return 1.01 * (decay_bound(g, complement) + 2.0 * U)


def _aged(a, step, b, s0, lengths, reverse=False):
    """Per element: S = the recurrence over |b| and |s0|, W = the same sum with
    every term times what its decays are off by."""
    S, W = np.zeros_like(b), np.zeros_like(b)
    start = 0
    fin_s, fin_w = np.zeros((len(lengths), b.shape[1])), np.zeros((len(lengths), b.shape[1]))
    for n, L in enumerate(lengths):
        s, w = np.abs(s0[n]).astype(np.float64), np.zeros(b.shape[1])
        order = range(start + L - 1, start - 1, -1) if reverse else range(start, start + L)
        for t in order:
            if reverse:          # lam = |dh| + mu: kept before the decay
                s = s + np.abs(b[t])
                S[t], W[t] = s, w
                s, w = a[t] * s, a[t] * (w + step[t] * s)
            else:
                s, w = a[t] * s + np.abs(b[t]), a[t] * (w + step[t] * s)
                S[t], W[t] = s, w
        fin_s[n], fin_w[n] = s, w
        start += L
    return S, W, fin_s, fin_w


def forward_bound(x, g, lengths, h0=None, complement=False):
    """Elementwise bounds of |h - fp32 h| and |s_final - fp32 s_final|."""
    step = _step(g, complement)
    x, a, gain = _parts(x, g, complement)
    z = np.zeros((len(lengths), x.shape[1])) if h0 is None else np.asarray(h0, np.float64)
    S, W, fs, fw = _aged(a, step, gain * x, z, lengths)
    return W + ENDS * S + 1e-36, fw + ENDS * fs + 1e-36


def backward_bound(x, g, lengths, d_h, h0=None, ds_final=None, complement=False):
    """Elementwise bounds of an fp32 (dx, dg, dh0)."""
    eh, _ = forward_bound(x, g, lengths, h0, complement)
    h, _ = forward(x, g, lengths, h0, complement)
    step = _step(g, complement)
    x, a, gain = _parts(x, g, complement)
    D = x.shape[1]
    z = np.zeros((len(lengths), D))
    S, W, fs, fw = _aged(a, step, np.asarray(d_h, np.float64),
                         z if ds_final is None else np.asarray(ds_final, np.float64), lengths,
                         reverse=True)
    elam = W + ENDS * S
    edx = np.abs(gain) * (elam + ENDS * S)
    hp, ehp = np.zeros_like(h), np.zeros_like(h)
    start = 0
    for n, L in enumerate(lengths):
        if L:
            hp[start] = 0.0 if h0 is None else h0[n]
            hp[start + 1:start + L] = h[start:start + L - 1]
            ehp[start + 1:start + L] = eh[start:start + L - 1]
        start += L
    mu, emu = a * S, a * (elam + (ENDS + step) * S)
    size = np.abs(hp) + (np.abs(x) if complement else 0.0)
    edg = emu * (size + ehp) + mu * (ehp + 3 * U * size)
    return edx + 1e-36, edg + 1e-36, fw + ENDS * fs + 1e-36
