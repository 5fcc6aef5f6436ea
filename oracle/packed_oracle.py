"""fp64 restatement of what a rounded layer meets after the solve: the 4-bit layout, its product with
activations, the 8-bit norm and the distillation loss. Plain numpy from the formulas of
``include/bakron.h``; shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

__all__ = ["pack4_layout", "matvec4", "rms_norm_q8", "distill"]


def _group_of(n, group_size):
    g = n if group_size is None else min(int(group_size), n)
    return np.arange(n) // g, -(-n // g)


def pack4_layout(codes, scales, group_size=None) -> np.ndarray:
    """The bytes of the 4-bit layout, entry by entry from its description."""
    codes = np.asarray(codes)
    m, n = codes.shape
    _, G = _group_of(n, group_size)
    scales = np.asarray(scales, dtype=np.float32).reshape(m, G)
    mt, kt = -(-m // 16), -(-n // 64)
    tiles = np.zeros(mt * kt * 512, dtype=np.uint8)
    for i in range(m):
        for j in range(n):
            r, c, t, h = i % 16, j % 8, (j % 32) // 8, (j % 64) // 32
            nib = int(f"{c:03b}"[::-1], 2)
            at = (i // 16 * kt + j // 64) * 512 + 16 * (4 * (r % 8) + t) + 8 * h + 4 * (r // 8)
            tiles[at + nib // 2] |= (int(codes[i, j]) & 15) << (4 * (nib % 2))
    steps = np.zeros((mt, G, 8, 2), dtype=np.float32)
    for i in range(m):
        steps[i // 16, :, i % 8, (i % 16) // 8] = scales[i]
    return np.concatenate([tiles, steps.reshape(-1).view(np.uint8)])


def matvec4(codes, scales, x, group_size=None, codebook=None, x_scales=None, x_group_size=None):
    """(y, a): y = x W^T and a = |x| |W|^T, the scale of its rounding errors."""
    codes = np.asarray(codes)
    m, n = codes.shape
    grp, G = _group_of(n, group_size)
    v = codes.astype(np.float64) if codebook is None else \
        np.asarray(codebook, dtype=np.float32).astype(np.float64)[codes]
    W = v * np.asarray(scales, dtype=np.float64).reshape(m, G)[:, grp]
    x = np.atleast_2d(np.asarray(x, dtype=np.float64))
    if x_scales is not None:
        gx, Gx = _group_of(n, x_group_size)
        x = x * np.asarray(x_scales, dtype=np.float64).reshape(x.shape[0], Gx)[:, gx]
    return x @ W.T, np.abs(x) @ np.abs(W).T


def rms_norm_q8(x, weight=None, eps=1e-6, residual=None, group_size=None):
    """(q, scales, h) per row."""
    x = np.atleast_2d(np.asarray(x, dtype=np.float64))
    h = x if residual is None else x + np.atleast_2d(np.asarray(residual, dtype=np.float64))
    rows, n = h.shape
    v = h if weight is None else h * np.asarray(weight, dtype=np.float64)
    rho = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    grp, G = _group_of(n, group_size)
    top = np.zeros((rows, G))
    for g in range(G):
        top[:, g] = np.abs(v[:, grp == g]).max(axis=1)
    full = top[:, grp]
    q = np.where(full > 0, np.rint(127.0 * v / np.where(full > 0, full, 1.0)), 0.0)
    return q.astype(np.int8), top * rho[:, None] / 127.0, h


def distill(z, top_idx, top_logits, tau=1.0, teacher_lse=None, row_weights=None):
    """(loss, lse, dz) per row."""
    z = np.atleast_2d(np.asarray(z, dtype=np.float64))
    rows, V = z.shape
    idx = np.asarray(top_idx).reshape(rows, -1)
    t = np.asarray(top_logits, dtype=np.float64).reshape(rows, -1)
    loss, lse, dz = np.zeros(rows), np.zeros(rows), np.zeros((rows, V))
    for r in range(rows):
        w = 1.0 if row_weights is None else float(row_weights[r])
        if w == 0.0:
            continue
        zr = z[r] / tau
        zmax = zr.max()
        lse[r] = zmax + np.log(np.exp(zr - zmax).sum())
        here = [(int(i), float(v) / tau) for i, v in zip(idx[r], t[r])
                if 0 <= i < V and v != -np.inf]
        if not here:
            continue
        tv = np.array([v for _, v in here])
        T = tv.max() + np.log(np.exp(tv - tv.max()).sum()) if teacher_lse is None \
            else float(teacher_lse[r])
        p = np.exp(tv - T)
        dz[r] = p.sum() * np.exp(zr - lse[r])
        for (i, v), pj in zip(here, p):
            if pj > 0:
                loss[r] += w * pj * ((v - T) - (zr[i] - lse[r]))
            dz[r, i] -= pj
        dz[r] *= w / tau
    return loss, lse, dz
