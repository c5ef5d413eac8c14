"""Plain float64 forms of the operators between the GEMMs of a layer: few-row products with an
NVFP4 weight, the residual norm with its gradient, rotary positions with several axes. Written from
the formulas with numpy, without any of the CUDA path's code."""
from __future__ import annotations

import numpy as np

from . import nvfp4_oracle as o


def gemv(x, codes, scales, G, bias=None, silu=False):
    """x (M x K) times the NVFP4 weight with element codes (N x K) and block-scale codes
    (N x K / 16). Returns the result and sum_k |x w|, the size that float32 sums' errors scale with."""
    x = np.asarray(x, np.float64)
    if silu:
        with np.errstate(over="ignore"):
            x = x / (1.0 + np.exp(-x))
    w = o.dequantize(codes, scales, 1.0).astype(np.float64) * float(G)
    y = x @ w.T
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, np.abs(x) @ np.abs(w).T


def sequences(rows, batches, offsets=None):
    """Sequence of each row, -1 where it has none."""
    b = np.full(rows, -1, np.int64)
    for i in range(batches):
        lo, hi = (i * rows // batches, (i + 1) * rows // batches) if offsets is None else offsets[i:i + 2]
        b[max(0, lo):max(0, hi)] = i
    return b


def _at(v, b, default):
    """Row b of a modulation tensor for every row, or the default."""
    return default if v is None else np.asarray(v, np.float64)[np.maximum(b, 0)]


def branch(y, post_norm=False, w_post=None, eps=1e-6):
    y = np.asarray(y, np.float64)
    if post_norm:
        y = y / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        if w_post is not None:
            y = y * np.asarray(w_post, np.float64)
    return y


def residual(x, y, b, gate=None, post_norm=False, w_post=None, residual_scale=1.0, eps=1e-6):
    """The stream after the branch is added."""
    return residual_scale * np.asarray(x, np.float64) + _at(gate, b, 1.0) * branch(y, post_norm, w_post, eps)


def stats(x, norm, eps=1e-6):
    x = np.asarray(x, np.float64)
    mean = x.mean(1, keepdims=True) if norm == "layer" else np.zeros((x.shape[0], 1))
    return mean, 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)


def modulated_norm(x, b, norm="layer", w=None, scale=None, shift=None, eps=1e-6):
    """The norm of the stored stream x, modulated."""
    mean, rstd = stats(x, norm, eps)
    n = (np.asarray(x, np.float64) - mean) * rstd
    if w is not None:
        n = n * np.asarray(w, np.float64)
    return n * (1.0 + _at(scale, b, 0.0)) + _at(shift, b, 0.0)


def residual_norm_backward(x_out, b, batches, dx_out=None, dh=None, y=None, gate=None, post_norm=False, w_post=None,
                           residual_scale=1.0, norm="layer", w=None, scale=None, eps=1e-6):
    """Gradients by the formulas. Returns a dict with dx, dy, dgate, dscale, dshift, dw, dw_post, and
    under "size_" + name what their float32 rounding errors scale with (sums of magnitudes)."""
    x_out = np.asarray(x_out, np.float64)
    rows, cols = x_out.shape
    live = (b >= 0)[:, None]
    t, size_t = np.zeros((rows, cols)), np.zeros((rows, cols))
    if dx_out is not None:
        t = np.asarray(dx_out, np.float64).copy()
        size_t = np.abs(t)
    out = {}
    onehot = (b[None, :] == np.arange(batches)[:, None]).astype(np.float64)
    if dh is not None:
        dh = np.asarray(dh, np.float64)
        mean, rstd = stats(x_out, norm, eps)
        xhat = (x_out - mean) * rstd
        wv = 1.0 if w is None else np.asarray(w, np.float64)
        one = 1.0 + _at(scale, b, 0.0)
        d = dh * one * wv
        m1 = d.mean(1, keepdims=True) if norm == "layer" else 0.0
        t = t + rstd * (d - m1 - xhat * (d * xhat).mean(1, keepdims=True))
        size_t = size_t + rstd * (np.abs(d) + np.abs(d).mean(1, keepdims=True)
                                  + np.abs(xhat) * np.abs(d * xhat).mean(1, keepdims=True))
        out["dshift"], out["size_dshift"] = onehot @ dh, onehot @ np.abs(dh)
        out["dscale"], out["size_dscale"] = onehot @ (dh * xhat * wv), onehot @ np.abs(dh * xhat * wv)
        v = np.where(live, dh * one * xhat, 0.0)
        out["dw"], out["size_dw"] = v.sum(0), np.abs(v).sum(0)
    out["dx"], out["size_dx"] = residual_scale * t, abs(residual_scale) * size_t
    if y is not None:
        yf = np.asarray(y, np.float64)
        g = _at(gate, b, 1.0)
        wp = 1.0 if w_post is None else np.asarray(w_post, np.float64)
        ry = 1.0 / np.sqrt((yf * yf).mean(1, keepdims=True) + eps) if post_norm else 1.0
        yh = yf * ry
        a = g * wp
        if post_norm:
            dy = ry * (a * t - yh * (a * t * yh).mean(1, keepdims=True))
            size = ry * (np.abs(a) * size_t + np.abs(yh) * (np.abs(a * yh) * size_t).mean(1, keepdims=True))
        else:
            dy, size = g * t, np.abs(g) * size_t
        out["dy"], out["size_dy"] = dy, size
        out["dgate"], out["size_dgate"] = onehot @ (t * yh * wp), onehot @ np.abs(size_t * yh * wp)
        v = np.where(live, g * t * yh, 0.0)
        out["dw_post"], out["size_dw_post"] = v.sum(0), np.where(live, np.abs(g * yh) * size_t, 0.0).sum(0)
    return out


def rope(x, positions, freqs, pairs, interleaved=True, inverse=False):
    """x: rows x heads x head_dim. Each pair as a complex number, turned by exp(i angle)."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    n = int(sum(pairs))
    axis = np.repeat(np.arange(len(pairs)), pairs)
    angle = np.asarray(positions, np.float64)[:, axis] * np.asarray(freqs, np.float64)[None, :]
    turn = np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    i = np.arange(n)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    z = (x[..., lo] + 1j * x[..., hi]) * turn
    out[..., lo], out[..., hi] = z.real, z.imag
    return out
