"""Float64 oracle of the block norms (numpy, written from the formulas).

    N(v; w)[t, c] = v[t, c] * rstd_t * (w_offset + w[c]),
    rstd_t = 1 / sqrt(mean_c v[t, c]^2 + eps)
    out = res_scale * x + gate * N(y; w_post);  h_next = N(out; w_next)

Where a stored tensor is read again (y by the post norm, out by the next
norm) the caller passes the stored values.  A gate is None, [T] (per token),
[H] (per channel) or [T, H]; `kind` tells the first two apart when T = H.
Every gradient comes with the sum of the absolute values of the terms it is
made of, which bounds the rounding error of a float32 evaluation.
"""
from __future__ import annotations

import numpy as np


def rstd(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1) + eps)


def norm(v, w, eps, w_offset=0.0):
    return v * rstd(v, eps)[:, None] * (w_offset + w)


def spread(gate, kind):
    """The gate as an array that broadcasts against [T, H]."""
    if kind == "none":
        return 1.0
    return gate[:, None] if kind == "token" else gate


def block_out(x, y, w_post, gate, kind, eps, w_offset=0.0, res_scale=1.0):
    """(out, the sum of absolute terms of out)."""
    n = y if w_post is None else norm(y, w_post, eps, w_offset)
    g = spread(gate, kind)
    return res_scale * x + g * n, np.abs(res_scale * x) + np.abs(g * n)


def norm_backward(v, w, dh, eps, w_offset=0.0):
    """(dv, dw, magnitude of dv, magnitude of dw) of <dh, N(v; w)>."""
    r = rstd(v, eps)[:, None]
    vh, dn = v * r, dh * (w_offset + w)
    dv = r * (dn - vh * np.mean(dn * vh, axis=1, keepdims=True))
    mv = r * (np.abs(dn) + np.abs(vh) * np.mean(np.abs(dn * vh), axis=1,
                                                keepdims=True))
    return dv, (dh * vh).sum(0), mv, np.abs(dh * vh).sum(0)


def block_out_backward(y, w_post, gate, kind, out, w_next, dout, dh, eps,
                       w_offset=0.0, res_scale=1.0):
    """{name: (gradient, magnitude)} of <dout, out> + <dh, N(out; w_next)>."""
    got = {}
    do, mo = np.zeros_like(y), np.zeros_like(y)
    if dh is not None:
        do, dwn, mo, mwn = norm_backward(out, w_next, dh, eps, w_offset)
        got["dw_next"] = (dwn, mwn)
    elif w_next is not None:
        got["dw_next"] = (np.zeros(y.shape[1]), np.zeros(y.shape[1]))
    if dout is not None:
        do, mo = do + dout, mo + np.abs(dout)
    got["dx"] = (res_scale * do, np.abs(res_scale) * mo)
    g = spread(gate, kind)
    dn, mn = do * g, mo * np.abs(g)
    if w_post is None:
        n = y
        got["dy"] = (dn, mn)
    else:
        n = norm(y, w_post, eps, w_offset)
        r = rstd(y, eps)[:, None]
        yh, wp = y * r, w_offset + w_post
        dy = r * (dn * wp - yh * np.mean(dn * wp * yh, axis=1,
                                         keepdims=True))
        my = r * (mn * np.abs(wp) + np.abs(yh) * np.mean(
            mn * np.abs(wp * yh), axis=1, keepdims=True))
        got["dy"] = (dy, my)
        got["dw_post"] = ((dn * yh).sum(0), (mn * np.abs(yh)).sum(0))
    if kind != "none":
        axis = {"token": 1, "channel": 0}.get(kind)
        dg, mg = do * n, mo * np.abs(n)
        got["dgate"] = (dg, mg) if axis is None else (dg.sum(axis),
                                                      mg.sum(axis))
    return got
