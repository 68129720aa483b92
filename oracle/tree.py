"""Drafted tokens over the paged cache, as plain float64 definitions (test infrastructure).

* ``rotate``: rotary positions. Pair (x, y) of a head turns by a = position * inv_freq[i]:
  (x cos a - y sin a, y cos a + x sin a) * magnitude, over pairs (i, i + R/2) or (2i, 2i + 1) of the
  first R elements; the others pass.
* ``attend_paged``: row i of sequence s (n_s drafted nodes at the end of a context of c_s tokens) sees
  the first c_s - n_s tokens and the nodes that its mask names:
  out = softmax(cap(scale * q.K)) V over what it sees, zeros where it sees nothing.
* ``commit``: rows of the accepted path move to the front of the drafted region.

The float64 angle of a float32 frequency and a position below 2^29 is exact to 2^-53 of itself.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import numpy as np

from . import attention


def rotate(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, interleaved: bool = False,
           magnitude: float = 1.0) -> np.ndarray:
    """x [T, H, D] (any float) -> float64 [T, H, D], rotated by each token's position."""
    out = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for t, pos in enumerate(np.asarray(positions).tolist()):
        for i, f in enumerate(np.asarray(inv_freq, dtype=np.float64).tolist()):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = magnitude * np.cos(pos * f), magnitude * np.sin(pos * f)
            u, v = np.array(x[t, :, a], dtype=np.float64), np.array(x[t, :, b], dtype=np.float64)
            out[t, :, a] = u * c - v * s
            out[t, :, b] = v * c + u * s
    return out


def visible(n: int, ctx: int, node: int, mask: Optional[int]) -> np.ndarray:
    """Which of the context's tokens a node sees. ``mask`` None is a chain."""
    start = ctx - n
    seen = np.zeros(ctx, dtype=bool)
    seen[:start] = True
    for j in range(n):
        seen[start + j] = j <= node if mask is None else bool(mask >> j & 1)
    return seen


def attend_paged(q: np.ndarray, k_pool: np.ndarray, v_pool: np.ndarray, block_tables: np.ndarray,
                 query_start: Sequence[int], context_lens: Sequence[int], masks: Optional[List[int]], scale: float,
                 num_kv_heads: int, kv_dtype: str, softcap: float = 0.0, k_scale: float = 1.0, v_scale: float = 1.0):
    """(out, weight) float64 [T, Hq, D]: the outputs, and sum_t softmax_t |V_t| (what roundings scale with)."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    G = Hq // num_kv_heads
    out, weight = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for s in range(len(context_lens)):
        r0, r1, ctx = int(query_start[s]), int(query_start[s + 1]), int(context_lens[s])
        for hk in range(num_kv_heads):
            K = attention.gather_context(k_pool, block_tables[s], ctx, hk, kv_dtype, k_scale)
            V = attention.gather_context(v_pool, block_tables[s], ctx, hk, kv_dtype, v_scale)
            for i in range(r1 - r0):
                seen = visible(r1 - r0, ctx, i, None if masks is None else masks[r0 + i])
                if not seen.any():
                    continue
                Ks, Vs = K[seen], V[seen]
                for h in range(hk * G, (hk + 1) * G):
                    x = float(scale) * (Ks @ q[r0 + i, h])
                    if softcap:
                        x = softcap * np.tanh(x / softcap)
                    w = np.exp(x - x.max())
                    out[r0 + i, h] = (w @ Vs) / w.sum()
                    weight[r0 + i, h] = (w @ np.abs(Vs)) / w.sum()
    return out, weight


def commit(k_pool: np.ndarray, v_pool: np.ndarray, block_tables: np.ndarray, query_start: Sequence[int],
           context_lens: Sequence[int], paths: Sequence[Sequence[int]], block_size: int = 16):
    """(k_pool, v_pool, lengths) after each sequence keeps its accepted path; pools of any row type."""
    k_out, v_out, lens = k_pool.copy(), v_pool.copy(), []
    for s, path in enumerate(paths):
        n = int(query_start[s + 1]) - int(query_start[s])
        start = int(context_lens[s]) - n
        for i, node in enumerate(path):
            a, b = start + node, start + i
            src, dst = int(block_tables[s][a // block_size]), int(block_tables[s][b // block_size])
            k_out[dst, :, b % block_size] = k_pool[src, :, a % block_size]
            v_out[dst, :, b % block_size] = v_pool[src, :, a % block_size]
        lens.append(start + len(path))
    return k_out, v_out, lens
