"""Float64 norms before and after the layer, with the block's gate, residual
scale and residual sum, and their vector-Jacobian product.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the
product path.

For a row of D channels, rms(x) = sqrt(mean(x^2) + eps):
    n     = o / rms(o) * w_post           (n = o without w_post)
    r_out = r + scale * sg(gate) * n
    h     = r_out / rms(r_out) * w_next

Pinned in ``tests/test_oracle_block_norm.py``: loops over single elements and
central finite differences.
"""

import numpy as np


def _logistic(a):
    t = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0, t) / (1.0 + t)


def block_norm(r, w_next, eps, o=None, gate=None, scale=None, w_post=None):
    """(r_out, h, rstd_post, rstd_next) in float64; None for what is absent
    (r_out without o, h and rstd_next without w_next, rstd_post without
    w_post)."""
    x, h, rp, rn = np.asarray(r, np.float64), None, None, None
    if o is not None:
        n = np.asarray(o, np.float64)
        if w_post is not None:
            rp = 1.0 / np.sqrt(np.mean(n * n, axis=-1) + eps)
            n = n * rp[..., None] * w_post
        if gate is not None:
            n = n * _logistic(np.asarray(gate, np.float64))
        if scale is not None:
            n = n * scale
        x = x + n
    if w_next is not None:
        rn = 1.0 / np.sqrt(np.mean(x * x, axis=-1) + eps)
        h = x * rn[..., None] * w_next
    return (x if o is not None else None), h, rp, rn


def _rms_vjp(x, rstd, w, dy):
    """(dx, dw) of y = x rstd w, rstd = 1 / sqrt(mean(x^2) + eps)."""
    D = x.shape[-1]
    t = dy * w
    dx = rstd[..., None] * t - x * (rstd ** 3 * np.sum(t * x, axis=-1) / D)[..., None]
    return dx, np.sum((dy * x * rstd[..., None]).reshape(-1, D), axis=0)


def block_norm_vjp(dr_out, dh, r_out, rstd_next, w_next, o=None, gate=None, scale=None, w_post=None,
                   rstd_post=None):
    """Gradients of block_norm's inputs given those of (r_out, h), as a dict
    with keys dr, do, dgate, dscale, dw_post, dw_next (absent ones missing)."""
    got = {}
    G = 0.0 if dr_out is None else np.asarray(dr_out, np.float64)
    if w_next is not None:
        dx, got["dw_next"] = _rms_vjp(np.asarray(r_out, np.float64), np.asarray(rstd_next, np.float64),
                                      np.asarray(w_next, np.float64), np.asarray(dh, np.float64))
        G = G + dx
    got["dr"] = G
    if o is None:
        return got
    o = np.asarray(o, np.float64)
    D = o.shape[-1]
    y = o * np.asarray(rstd_post, np.float64)[..., None] * w_post if w_post is not None else o
    u = _logistic(np.asarray(gate, np.float64)) if gate is not None else np.ones_like(o)
    c = np.asarray(scale, np.float64) if scale is not None else np.ones(D)
    if gate is not None:
        got["dgate"] = G * c * y * u * (1.0 - u)
    if scale is not None:
        got["dscale"] = np.sum((G * u * y).reshape(-1, D), axis=0)
    dy = G * c * u
    if w_post is not None:
        got["do"], got["dw_post"] = _rms_vjp(o, np.asarray(rstd_post, np.float64),
                                             np.asarray(w_post, np.float64), dy)
    else:
        got["do"] = dy
    return got
