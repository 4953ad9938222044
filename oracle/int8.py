"""Oracle for the int8 GEMM with token and channel scales: the integer sum exactly, the rest in FP64.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product library; it shares no
code with the CUDA path.

  D[i][j] = relu?( sum_k a_ik b_jk * row_scale[i] * col_scale[j] + bias[j] )

grouped: rows r_g .. r_g + M_g - 1 of A and D belong to group g, whose B, col_scale and bias are its part of
groups * N rows or elements.
"""
from __future__ import annotations

import numpy as np


def sums(A, B):
    """sum_k a_ik b_jk as int64: FP64 holds every partial sum below 2^53 exactly."""
    s = np.asarray(A, dtype=np.float64) @ np.asarray(B, dtype=np.float64).T
    return s.astype(np.int64)


def gemm(A, B, row_scale, col_scale, bias=None, relu=False, group_rows=None):
    """D in FP64, and the magnitude of each element's product part."""
    A = np.asarray(A)
    if group_rows is None:
        group_rows, parts = [A.shape[0]], 1
    else:
        parts = len(group_rows)
    N = B.shape[0] // parts
    D = np.full((A.shape[0], N), np.nan)
    size = np.zeros((A.shape[0], N))
    at = 0
    for g, rows in enumerate(group_rows):
        here, mine = slice(at, at + rows), slice(g * N, (g + 1) * N)
        s = sums(A[here], B[mine]) * np.asarray(row_scale, dtype=np.float64)[here, None] * \
            np.asarray(col_scale, dtype=np.float64)[None, mine]
        size[here] = np.abs(s)
        if bias is not None:
            s = s + np.asarray(bias, dtype=np.float64)[None, mine]
        D[here] = np.maximum(s, 0.0) if relu else s
        at += rows
    return D, size
