"""fp64 CPU oracle for the operators around the paged attention: the norm, rotation and write
of new tokens, accumulated attention weights, eviction, and the linear layer.

TEST INFRASTRUCTURE ONLY. Nothing on the product path may import, call or run this module. It
shares no code with the CUDA path. Plain loops over sequences and heads, written from the
formulas; every function takes the exact values the GPU sees, widened to fp64.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rms_norm", "rotate", "append", "key_weights", "evict", "linear"]


def rms_norm(x, weight, eps):
    """``x / sqrt(mean(x^2) + eps) * weight`` over the last axis."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, angles, interleaved):
    """Turns pair p of the last axis by ``angles[..., p]`` (broadcast over the other axes)."""
    x = np.array(x, dtype=np.float64)
    n = angles.shape[-1]
    c, s = np.cos(angles), np.sin(angles)
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo] = a * c - b * s
    x[..., hi] = b * c + a * s
    return x


def append(q, k, v, k_pages, v_pages, block_table, prefix_lens, chunk_lens, positions, inv_freq, pair_axis, q_norm,
           k_norm, eps, interleaved, q_out):
    """The whole call on copies: ``(q_out, k_pages, v_pages)``. ``positions`` ``[axes, B, C]``."""
    q_out, k_pages, v_pages = (np.array(t, dtype=np.float64) for t in (q_out, k_pages, v_pages))
    page = k_pages.shape[2]
    B, C = q.shape[:2]
    pairs = 0 if inv_freq is None else len(inv_freq)
    for b in range(B):
        n = C if chunk_lens is None else int(chunk_lens[b])
        for i in range(n):
            at = int(prefix_lens[b]) + i
            angles = np.array([float(positions[0 if pair_axis is None else pair_axis[p]][b][i]) * float(inv_freq[p])
                               for p in range(pairs)])
            rows = []
            for x, w in ((q[b, i], q_norm), (k[b, i], k_norm)):
                y = np.asarray(x, dtype=np.float64) if w is None else rms_norm(x, w, eps)
                rows.append(rotate(y, angles, interleaved) if pairs else y)
            q_out[b, i] = rows[0]
            p = int(block_table[b][at // page])
            k_pages[p, :, at % page] = rows[1]
            v_pages[p, :, at % page] = v[b, i]
    return q_out, k_pages, v_pages


def key_weights(q, k_pages, block_table, lens, lse, scale, first=None, last=None):
    """``[B, Hkv, cap]``: the softmax weight each key receives from queries ``first .. last - 1``
    of each sequence (``q`` ``[B, C, Hq, D]``), query i seeing keys ``0 .. lens[b] + i``; slots
    past the sequence are NaN. ``lse`` ``[B, Hq, C]``."""
    q, k_pages, lse = (np.asarray(t, dtype=np.float64) for t in (q, k_pages, lse))
    B, C, Hq, _ = q.shape
    _, Hkv, page, _ = k_pages.shape
    cap = block_table.shape[1] * page
    out = np.full((B, Hkv, cap), np.nan)
    for b in range(B):
        lo, hi = (0 if first is None else int(first[b])), (C if last is None else int(last[b]))
        n = int(lens[b]) + hi
        for g in range(Hkv):
            keys = np.array([k_pages[int(block_table[b][t // page]), g, t % page] for t in range(n)]).reshape(n, k_pages.shape[3])
            total = np.zeros(n)
            for i in range(lo, hi):
                see = int(lens[b]) + i + 1
                for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                    total[:see] += np.exp(scale * (keys[:see] @ q[b, i, h]) - lse[b, h, i])
            out[b, g, :n] = total
    return out


def evict(kv_lens, sums, budget, n_sink, n_recent):
    """``(kept, new_lens, new_sums)``: lists of kept indices per (b, head), in order. NaN ranks
    above every number."""
    kept, lens, new = [], [], []
    for b, n in enumerate(int(x) for x in kv_lens):
        lens.append(min(n, budget))
        for row in np.asarray(sums)[b]:
            if n <= budget:
                keep = list(range(n))
            else:
                fixed = set(range(n_sink)) | set(range(n - n_recent, n))
                rest = [t for t in range(n) if t not in fixed]
                rest.sort(key=lambda t: (0 if math.isnan(row[t]) else 1, 0.0 if math.isnan(row[t]) else -row[t], t))
                keep = sorted(fixed | set(rest[:budget - len(fixed)]))
            kept.append(keep)
            new.append([float(row[t]) for t in keep])
    return kept, lens, new


def linear(x, w, bias=None, activation="none", residual=None):
    """``act(x w^T + bias) + residual``."""
    y = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    if activation == "relu":
        y = np.maximum(y, 0.0)
    elif activation == "gelu":
        y = 0.5 * y * (1.0 + np.vectorize(math.erf)(y * math.sqrt(0.5)))
    elif activation == "gelu_tanh":
        y = 0.5 * y * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
    elif activation == "silu":
        with np.errstate(over="ignore"):
            y = y / (1.0 + np.exp(-y))
    elif activation != "none":
        raise ValueError(activation)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)
