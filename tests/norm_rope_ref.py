"""The per-head norm and rotation of queries and keys, its sign-bit form and its
gradient in 64 bits, straight from the formulas, with the bounds that the
kernels' 32-bit arithmetic allows.

U = 2^-24 is half a step of fp32, relative. A row's sum of squares is added in
chains of at most d / 4 + 8 roundings and rsqrtf is good to 2 steps, so r is off
by at most (d / 8 + 8) U relative; y = x r w and its turn add a few roundings
more. K U with K = d / 4 + 32 covers each of them, relative to the sizes of the
products that are added (`size` below), which cancellation does not shrink. An
output in bf16 adds half a step of its value (2^-8 relative).
"""
import numpy as np
import torch

U = 2.0 ** -24


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def pairs(d, rot, inter):
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if inter else (p, p + rot // 2)


def tables(cos, sin, B):
    """[B, 1, N, rot / 2] float64."""
    c, s = f64(cos), f64(sin)
    if c.ndim == 2:
        c, s = np.broadcast_to(c, (B,) + c.shape), np.broadcast_to(s, (B,) + s.shape)
    return c[:, None], s[:, None]


def turn(y, c, s, inter, back=False, size=False):
    """y with its pairs turned (back: by minus the angles; size: the sum of the products' magnitudes)."""
    a, b = pairs(y.shape[-1], 2 * c.shape[-1], inter)
    if back:
        s = -s
    z = np.abs(y) if size else y.copy()
    if size:
        z[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
        z[..., b] = np.abs(y[..., a] * s) + np.abs(y[..., b] * c)
    else:
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., a] * s + y[..., b] * c
    return z


def forward(x, w, cos, sin, eps, inter):
    """(z, size) float64; x [B,H,N,d] numpy, w [d] or None, cos / sin torch or None."""
    d = x.shape[-1]
    w = np.ones(d) if w is None else f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * r * w
    if cos is None:
        return y, np.abs(y)
    c, s = tables(cos, sin, x.shape[0])
    return turn(y, c, s, inter), turn(y, c, s, inter, size=True)


def signs(x, w, cos, sin, inter):
    """[z >= 0] decided from x_a w_a cos - x_b w_b sin in 64 bits, products left to right."""
    w = np.ones(x.shape[-1]) if w is None else f64(w)
    u = x * w
    if cos is None:
        return u >= 0
    c, s = tables(cos, sin, x.shape[0])
    return turn(u, c, s, inter) >= 0


def words(on):
    d = on.shape[-1]
    W = (d + 31) // 32
    out = np.zeros(on.shape[:-1] + (W,), np.uint32)
    for ch in range(d):
        out[..., ch // 32] |= on[..., ch].astype(np.uint32) << np.uint32(ch % 32)
    return out


def backward(x, dz, w, cos, sin, eps, inter):
    """dx, its size, dw, its size (float64)."""
    d = x.shape[-1]
    w = np.ones(d) if w is None else f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    if cos is None:
        dy, sy = dz, np.abs(dz)
    else:
        c, s = tables(cos, sin, x.shape[0])
        dy, sy = turn(dz, c, s, inter, back=True), turn(dz, c, s, inter, size=True)
    g, sg = dy * w, sy * np.abs(w)
    mean = (g * xh).mean(-1, keepdims=True)
    smean = (sg * np.abs(xh)).mean(-1, keepdims=True)
    dx, sx = r * (g - xh * mean), r * (sg + np.abs(xh) * smean)
    ax = (0, 1, 2)
    return dx, sx, (dy * xh).sum(ax), (sy * np.abs(xh)).sum(ax)


def close(got, ref, size, d, dtype, what, steps=0):
    """|got - ref| <= K U size (+ steps U size: additions in a chain of that length) + half a step of the type."""
    g = f64(got)
    assert g.shape == ref.shape, what
    bound = (d / 4 + 32 + steps) * U * size
    if dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8
    bad = np.abs(g - ref) > bound + 1e-37
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, worst {np.abs(g - ref).max():.3e}"
