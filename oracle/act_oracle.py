"""Plain CPU definitions of the 8-bit activations, the RMSNorm and the embedding.

TEST INFRASTRUCTURE ONLY -- see the package docstring.  NumPy, fp64, written
from the formulas documented in ``include/forge.h``:

* 8-bit activations: per block of a row, ``a = max|x|``, ``Q`` = 127 (S8) or 448
  (E4M3), ``e`` the smallest integer >= -120 with ``a <= Q 2^e``; code = ``x 2^-e``
  to nearest, ties to even; stored value ``code 2^e``; scale byte ``e + 127``.  A
  block with a non-finite value: scale byte 255, codes 0, all values NaN.
* RMSNorm: ``h = x + r`` (rounded to r's format), ``s = 1 / sqrt(mean h^2 + eps)``,
  ``y = h s gamma``; backward ``dx = s (g - n mean(g n)) + dr`` with
  ``g = gamma dy``, ``n = h s``, and ``dgamma = sum dy n``.
* Embedding: ``y_t = scale W[id_t]``; ``G[v] = scale sum_{id_t = v} dy_t``; ids outside
  the vocabulary give zeros and take no gradient.
"""

from __future__ import annotations

import math

import numpy as np

from .forge_oracle import e4m3_to_f64, f32_to_e4m3_rne

__all__ = ["ACT8_QMAX", "ACT8_EMIN", "act8_exponent", "act8_encode", "act8_decode", "rmsnorm", "rmsnorm_backward",
           "embed", "embed_grad"]

ACT8_QMAX = {"s8": 127.0, "e4m3": 448.0}
ACT8_EMIN = -120


def act8_exponent(a: float, fmt: str) -> int:
    """The exponent of a block with absmax ``a`` (finite), by the definition: counted up from the smallest."""
    e = ACT8_EMIN
    while a > math.ldexp(ACT8_QMAX[fmt], e):
        e += 1
    return e


def act8_encode(x32: np.ndarray, fmt: str, block: int):
    """(codes, scale bytes) of a float32 matrix; codes int8 (S8) or uint8 (E4M3)."""
    x = np.asarray(x32, dtype=np.float32)
    rows, cols = x.shape
    nb = -(-cols // block)
    codes = np.zeros((rows, cols), np.int8 if fmt == "s8" else np.uint8)
    scale = np.zeros((rows, nb), np.uint8)
    qf, qe = math.frexp(ACT8_QMAX[fmt])
    for b in range(nb):
        part = x[:, b * block:(b + 1) * block].astype(np.float64)
        bad = ~np.isfinite(part).all(axis=1)
        part = np.where(bad[:, None], 0.0, part)
        af, ae = np.frexp(np.abs(part).max(axis=1))
        e = np.where(af == 0, ACT8_EMIN, np.maximum(ae - qe + (af > qf), ACT8_EMIN)).astype(np.int64)
        y = np.ldexp(part, -e[:, None])
        if fmt == "s8":
            c = np.rint(y).astype(np.int8)
        else:
            c = f32_to_e4m3_rne(y.astype(np.float32))
        codes[:, b * block:(b + 1) * block] = np.where(bad[:, None], c.dtype.type(0), c)
        scale[:, b] = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes, scale


def act8_decode(codes: np.ndarray, scale: np.ndarray, fmt: str, block: int) -> np.ndarray:
    """The stored values, fp64, exactly."""
    v = codes.astype(np.float64) if fmt == "s8" else e4m3_to_f64(codes)
    s = np.repeat(scale.astype(np.int64), block, axis=1)[:, :codes.shape[1]]
    return np.where(s == 255, np.nan, np.ldexp(v, (s - 127).astype(np.int32)))


def rmsnorm(h: np.ndarray, gamma: np.ndarray, eps: float):
    """(y, s) in fp64 of h [rows, cols], the sum as stored."""
    h = np.asarray(h, np.float64)
    s = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * s[:, None] * np.asarray(gamma, np.float64), s


def rmsnorm_backward(dy, h, gamma, rstd, dr=None):
    """(dx, dgamma, the sums of absolute values behind dx and dgamma) in fp64."""
    dy, h, gamma, s = (np.asarray(t, np.float64) for t in (dy, h, gamma, rstd))
    s = s[:, None]
    g, n = dy * gamma, h * s
    dx = s * (g - n * np.mean(g * n, axis=1, keepdims=True))
    dx_abs = s * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), axis=1, keepdims=True))
    if dr is not None:
        dx = dx + np.asarray(dr, np.float64)
        dx_abs = dx_abs + np.abs(np.asarray(dr, np.float64))
    return dx, np.sum(dy * n, axis=0), dx_abs, np.sum(np.abs(dy * n), axis=0)


def embed(ids, W, scale: float) -> np.ndarray:
    ids, W = np.asarray(ids), np.asarray(W, np.float64)
    ok = (ids >= 0) & (ids < W.shape[0])
    y = np.zeros((len(ids), W.shape[1]))
    y[ok] = W[ids[ok]] * scale
    return y


def embed_grad(ids, dy, V: int, scale: float):
    """(G, the same sum of absolute values, tokens per row)."""
    ids, dy = np.asarray(ids), np.asarray(dy, np.float64)
    G, A, n = np.zeros((V, dy.shape[1])), np.zeros((V, dy.shape[1])), np.zeros(V, np.int64)
    for t, v in enumerate(ids):
        if 0 <= v < V:
            G[v] += dy[t]
            A[v] += np.abs(dy[t])
            n[v] += 1
    return G * scale, A * abs(scale), n
