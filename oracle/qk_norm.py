"""fp64 norm of each head with the position rotation, and its gradients, written
from their formulas (include/gdn_qk_norm.h), with bounds of an fp32 evaluation.

One side (queries or keys) at a time: x [T, H, d] numpy; w [d] or None;
positions [T] and inv_freq [F] or None.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32


def _pairs(F, interleaved):
    j = np.arange(F)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + F)


def rotate(n, positions, inv_freq, interleaved, sign=1.0):
    if inv_freq is None:
        return n
    ang = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang)[:, None, :], sign * np.sin(ang)[:, None, :]
    i, k = _pairs(len(inv_freq), interleaved)
    y = n.copy()
    y[..., i] = n[..., i] * c - n[..., k] * s
    y[..., k] = n[..., k] * c + n[..., i] * s
    return y


def _mix(v, inv_freq, interleaved):
    """|v| of both channels of a rotated pair on each of them (what a rotation's
    result can be made of)."""
    v = np.abs(v)
    if inv_freq is None:
        return v
    i, k = _pairs(len(inv_freq), interleaved)
    y = v.copy()
    y[..., i] = y[..., k] = v[..., i] + v[..., k]
    return y


def _r(x, norm, eps):
    m = (x * x).sum(-1, keepdims=True)
    return 1.0 / np.sqrt((m / x.shape[-1] if norm == "rms" else m) + eps)


def forward(x, w=None, positions=None, inv_freq=None, *, norm="l2", eps=1e-6, interleaved=False):
    x = np.asarray(x, np.float64)
    n = x * _r(x, norm, eps)
    if w is not None:
        n = n * np.asarray(w, np.float64)
    return rotate(n, positions, inv_freq, interleaved)


def backward(x, dy, w=None, positions=None, inv_freq=None, *, norm="l2", eps=1e-6,
             interleaved=False):
    """Returns (dx, dw); dw is the gradient of a weight of ones when w is None."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    r = _r(x, norm, eps)
    dn = rotate(dy, positions, inv_freq, interleaved, -1.0)
    e = dn if w is None else dn * np.asarray(w, np.float64)
    m = (x * e).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1)
    return r * (e - x * r * r * m), (dn * x * r).sum((0, 1))


def forward_bound(x, w=None, positions=None, inv_freq=None, *, norm="l2", eps=1e-6,
                  interleaved=False):
    """Elementwise bound of an fp32 y.  The sum of squares: at most 11 roundings
    on a path (5 on a lane, 5 between lanes, eps), half of that in r, two units
    in the last place (4 U) of rsqrtf, two products: 11.5 U.  A rotation: cosine
    and sine are off by at most 3 U (one unit in the last place of sincospif, and
    the rounding of an angle below an eighth of a turn), product and sum 2 U."""
    n = np.asarray(x, np.float64) * _r(np.asarray(x, np.float64), norm, eps)
    if w is not None:
        n = n * np.asarray(w, np.float64)
    return 17 * U * _mix(n, inv_freq, interleaved) + 1e-36


def backward_bound(x, dy, w=None, positions=None, inv_freq=None, *, norm="l2", eps=1e-6,
                   interleaved=False):
    """Elementwise bounds of an fp32 (dx, dw).  With E the size of e: e is off by
    6 U E (rotation and weight), r by 9.5 U, m(x e) by 10 U + 6 U, r^2 m(x e) by
    19 U + 16 U and three products, its product with x and the difference by 2 U,
    and r once more by 10.5 U: 51 U.  dw: a term is off by 5 U + 10.5 U and a
    rounding, and a sum of K terms by at most K U of their sizes."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    r = _r(x, norm, eps)
    dn = _mix(dy, inv_freq, interleaved)
    e = dn if w is None else dn * np.abs(np.asarray(w, np.float64))
    m = (np.abs(x) * e).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1)
    terms = (dn * np.abs(x) * r).sum((0, 1))
    K = x.shape[0] * x.shape[1]
    return 51 * U * r * (e + np.abs(x) * r * r * m) + 1e-36, (17 + K) * U * terms + 1e-36
