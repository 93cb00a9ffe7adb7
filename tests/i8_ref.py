"""Plain numpy forms of the layer norm and of the 8-bit integer linear: every sum in 64 bits (integers exact), every
fp32 step rounded once, as include/nvfp4.h states them."""
import numpy as np

F = np.float32
HALF = 2.0 ** -24            # half a step of fp32, relative


def i8_quantize(v):
    """(codes int8, scales float32) of the rows of v, finite float32."""
    v = np.asarray(v, F)
    amax = np.abs(v).max(axis=1)
    zero = amax < F(2.0 ** -110)
    with np.errstate(divide="ignore", over="ignore"):
        scale = np.where(zero, F(0), amax / F(127)).astype(F)
        inv = np.where(zero, F(0), F(127) / amax).astype(F)
    return np.rint(v * inv[:, None]).astype(np.int8), scale


def layernorm(x, gamma=None, beta=None, eps=1e-5):
    """(y float32 before its last rounding, mean, rstd) of the rows of x, float32."""
    x = np.asarray(x, F)
    mean = (x.astype(np.float64).sum(axis=1) / x.shape[1]).astype(F)
    d = x - mean[:, None]
    var = (d.astype(np.float64) ** 2).sum(axis=1) / x.shape[1]
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = (1.0 / np.sqrt(var + np.float64(F(eps)))).astype(F)
        y = d * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, F)
    if beta is not None:
        y = y + np.asarray(beta, F)
    assert y.dtype == F
    return y, mean, rstd


def layernorm_backward(dy, x, mean, rstd, gamma=None):
    """Gradients in 64 bits from the given statistics: dx, dgamma, dbeta, and for each the sum of the magnitudes that
    go into it (what a rounding error of the fp32 sums is relative to)."""
    dy, x, mean, rstd = (np.asarray(a, np.float64) for a in (dy, x, mean, rstd))
    K = x.shape[1]
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    c1, c2 = g.sum(1, keepdims=True) / K, (g * xh).sum(1, keepdims=True) / K
    r = rstd[:, None]
    dx = r * (g - c1 - xh * c2)
    # |x| + |mean| covers the rounding of x - mean
    ax = np.abs(xh) + (np.abs(x) + np.abs(mean[:, None])) * r
    mx = r * (np.abs(g) + np.abs(g).sum(1, keepdims=True) / K + ax * (np.abs(g) * ax).sum(1, keepdims=True) / K)
    return (dx, (dy * xh).sum(0), dy.sum(0)), (mx, (np.abs(dy) * ax).sum(0), np.abs(dy).sum(0))


def i8_gemm(a, a_scales, w, w_scales, bias=None):
    """float32 result before the rounding to the output type."""
    acc = (a.astype(np.float64) @ w.astype(np.float64).T)       # integers below 2^31: exact in binary64
    y = acc.astype(F) * np.asarray(a_scales, F)[:, None] * np.asarray(w_scales, F)
    if bias is not None:
        y = y + np.asarray(bias, F)
    assert y.dtype == F
    return y
