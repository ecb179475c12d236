"""Plain fp64 definitions of the operators in front of the attention (numpy, row by row).

Test infrastructure only; shares no code with the kernels.  Inputs are numpy arrays whose
values are exactly those the kernels get (bf16 values widened), outputs are float64.
"""

from __future__ import annotations

import math

import numpy as np


def tree_positions(parent, cu, ctx, prefix_len, T, fill=0):
    """positions [T] int64; rows of no sequence hold `fill`.  parent None: chains."""
    out = np.full(T, fill, dtype=np.int64)
    for b in range(len(cu) - 1):
        start = prefix_len + (0 if ctx is None else int(ctx[b]))
        for t in range(cu[b + 1] - cu[b]):
            up = t - 1 if parent is None else int(parent[cu[b] + t])
            out[cu[b] + t] = start if up < 0 else out[cu[b] + up] + 1
    return out


def angles(positions, freq):
    """[T, R / 2] radians: the exact product of position and turns, less its whole turns."""
    turns = [[(int(p) * int(f)) % (1 << 64) for f in freq] for p in positions]
    return 2 * math.pi * (np.array(turns, dtype=object).astype(np.float64) / 2.0 ** 64).reshape(
        len(positions), len(freq))


def head_rows(x, w, positions, freq, interleaved, scale, norm, eps):
    """x [T, H, D] normalised and rotated; returns (y, a) with a = |x| + |y| of the pair that an
    element is rotated with (its own size where it is not), the size of the terms of y."""
    y = x.astype(np.float64)
    D = y.shape[2]
    if norm is not None:
        square = (y * y).sum(axis=2, keepdims=True)
        y = y / np.sqrt(square / (D if norm == "rms" else 1) + eps)
        if w is not None:
            y = y * w.astype(np.float64)
    size = np.abs(y)
    if freq is not None and len(freq):
        half = len(freq)
        a = angles(positions, freq)[:, None]
        i = np.arange(half)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        u, v = y[..., first], y[..., second]
        out = y.copy()
        out[..., first] = scale * (u * np.cos(a) - v * np.sin(a))
        out[..., second] = scale * (v * np.cos(a) + u * np.sin(a))
        size[..., first] = size[..., second] = abs(scale) * (np.abs(u) + np.abs(v))
        y = out
    return y, size


def append_positions(cu, ctx, prefix_len, T):
    """Row numbers of the cache [T] and positions [T] of every sequence's rows (-1: no row)."""
    at = np.full(T, -1, dtype=np.int64)
    for b in range(len(cu) - 1):
        at[cu[b]:cu[b + 1]] = int(ctx[b]) + np.arange(cu[b + 1] - cu[b])
    return at, np.where(at < 0, 0, at + prefix_len)


def place(cache, rows, cu, table, ctx):
    """The cache after the rows of each sequence were put behind its context."""
    cache, page = np.array(cache, dtype=np.float64), cache.shape[1]
    for b in range(len(cu) - 1):
        for j in range(cu[b + 1] - cu[b]):
            p = int(ctx[b]) + j
            cache[table[b][p // page], p % page] = rows[cu[b] + j]
    return cache


def frequencies(R, base, stretch=None, factor=1.0, trained_len=0.0, fast=32.0, slow=1.0):
    """(radians a position [R / 2], scale), in extended precision where numpy has it."""
    L = np.longdouble
    i = np.arange(R // 2).astype(L)
    if stretch == "ntk":
        base = L(base) * L(factor) ** (L(R) / L(R - 2))
    f = L(base) ** (-2 * i / L(R))
    if stretch == "linear":
        return f / L(factor), 1.0
    if stretch in ("yarn", "bands"):
        turns = L(trained_len) * f / (2 * np.pi)
        if stretch == "bands":
            keep = np.clip((turns - slow) / (L(fast) - L(slow)), 0, 1)
            return keep * f + (1 - keep) * f / factor, 1.0

        def pair(n):
            return R * math.log(trained_len / (2 * math.pi * n)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
        # (all pairs turn fewer than `slow` times, or all more than `fast`: no blend)
        late = np.clip((i - lo) / (hi - lo), 0, 1) if hi > lo else (i >= hi).astype(L)
        return (1 - late) * f + late * f / factor, 0.1 * math.log(factor) + 1
    return f, 1.0
