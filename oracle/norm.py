"""Residual addition and root-mean-square norm in float64 (oracle; test infrastructure)."""
import numpy as np


def rms_norm(r, weight, eps):
    """Rows r / sqrt(mean(r^2) + eps) * weight; ``r`` as the sum was rounded."""
    r = np.asarray(r, np.float64)
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def scales_of(y, group=0):
    """max |y| / 448 of each row or of each group of values."""
    rows, n = y.shape
    return np.abs(y).reshape(rows, -1, group or n).max(2) / 448.0
