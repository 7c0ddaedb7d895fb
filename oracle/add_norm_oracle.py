"""Float64 oracle of the residual norm, its 8-bit forms and its gradients, in
numpy."""
import numpy as np

from oracle.norm_rope_oracle import round_bf16


def add(x, residual):
    """The sum rounded to bf16 (x itself without a residual)."""
    return x if residual is None else round_bf16(x + residual)


def norm(z, weight, eps):
    """Unrounded normed rows."""
    return z / np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps) * weight


E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def codes(y, size):
    """(values of the e4m3 codes, scales) of bf16 rows y [n, d], one scale for
    each `size` values: the smallest power of two that brings the largest to at
    most 448; codes nearest, ties to the even one."""
    n, d = y.shape
    values, scales = np.empty_like(y), np.ones((n, -(-d // size)))
    for g in range(scales.shape[1]):
        t = y[:, g * size:(g + 1) * size]
        for r in range(n):
            top = np.abs(t[r]).max()
            k = -64
            while top > 448 * 2.0 ** k and k < 31:
                k += 1
            scales[r, g] = 2.0 ** k if top > 0 else 1.0
        x = np.abs(t) / scales[:, g:g + 1]
        up = np.clip(np.searchsorted(E4M3, x), 1, len(E4M3) - 1)
        lo, hi = E4M3[up - 1], E4M3[up]
        down = (x - lo < hi - x) | ((x - lo == hi - x) & (up % 2 == 1))
        values[:, g * size:(g + 1) * size] = np.copysign(np.where(down, lo, hi), t)
    return values, scales


def grads(z, weight, eps, dout, dresidual=None):
    """(dx, dweight, the sums of the magnitudes of their terms)."""
    r = 1 / np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps)
    zh, g = z * r, weight * dout
    dx = r * (g - zh * np.mean(g * zh, axis=-1, keepdims=True))
    size = r * (np.abs(g) + np.abs(zh) * np.mean(np.abs(g * zh), axis=-1, keepdims=True))
    if dresidual is not None:
        dx, size = dx + dresidual, size + np.abs(dresidual)
    return dx, np.sum(dout * zh, axis=0), size, np.sum(np.abs(dout * zh), axis=0)
