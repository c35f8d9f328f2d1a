"""ORACLE -- test infrastructure only (tests).

Reference for the query / key / value writer in numpy fp64, one token and head at a time, as
include/hpa.h states it; beside each value the magnitude M that fp32 errors scale with.
"""
from __future__ import annotations

import math

import numpy as np

from .feeder import hadamard

D = 128


def head(x, pos, cos_sin, w, eps, norm_after, interleaved, use_hadamard):
    """(row, M): a query's or key's 128 values after norm, rotation and transform."""
    x = np.asarray(x, np.float64).copy()

    def norm(y):
        return y if w is None else y / math.sqrt(np.mean(y * y) + eps) * np.asarray(w, np.float64)

    if not norm_after:
        x = norm(x)
    size = np.abs(x)
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        half = rot // 2
        c, s = np.asarray(cos_sin[pos, :half], np.float64), np.asarray(cos_sin[pos, half:], np.float64)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            size[a], size[b] = (abs(x[a] * c[i]) + abs(x[b] * s[i]),
                                abs(x[b] * c[i]) + abs(x[a] * s[i]))
            x[a], x[b] = x[a] * c[i] - x[b] * s[i], x[b] * c[i] + x[a] * s[i]
    if norm_after:
        y = norm(x)
        with np.errstate(divide="ignore", invalid="ignore"):
            size = np.where(x != 0, size * np.abs(y / np.where(x != 0, x, 1)), size)
        x = y
    if use_hadamard:
        return hadamard(D) @ x, np.full(D, size.sum() / math.sqrt(D))
    return x, size
