"""Plain 64-bit (or exact) definitions of the operators around a step's attention
-- TEST INFRASTRUCTURE ONLY, like the rest of this package.

Each is written from the definition in the header of the C ABI; nothing here
shares code with the library.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch


def _f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, axis_map=None, interleaved=False):
    """Heads x [N, H, D] normed (with a weight) and rotated: (values, size of the
    rotated pair each belongs to), both [N, H, D]."""
    y = _f64(x).copy()
    N, H, D = y.shape
    if weight is not None:
        y /= np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        y *= _f64(weight)
    f = _f64(inv_freq)
    F = f.size
    pos = positions.cpu().numpy().reshape(-1, N).astype(np.int64)
    axis = np.zeros(F, dtype=np.int64) if axis_map is None else axis_map.cpu().numpy()
    size = np.abs(y)
    for i in range(F):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + F)
        angle = pos[axis[i]].astype(np.float64) * f[i]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        size[..., a] = size[..., b] = np.hypot(u, v)
    return y, size


def _probability(v: float) -> Fraction:
    if not v > 0.0:                                  # NaN too
        return Fraction(0)
    return Fraction(min(v, 1.0))


def verify(tokens, parents, target, uniforms, draft=None, draft_lens=None, max_path=None):
    """(path, path_lens, next_tokens) as lists, in exact arithmetic."""
    B, T = tokens.shape
    extra = target.shape[1] - T
    V = target.shape[2]
    A = T if max_path is None else max_path
    paths, lens, drawn = [], [], []
    for b in range(B):
        d = T if draft_lens is None else max(0, min(T, int(draft_lens[b])))
        par = [int(parents[b, t]) for t in range(d)]
        par = [x if -1 <= x < t else -1 for t, x in enumerate(par)]
        u = [Fraction(min(max(float(x), 0.0), 1.0)) if x == x else None for x in uniforms[b].tolist()]

        def row(of, node):
            return [_probability(x) for x in of[b, node + extra].tolist()]

        path, node, start = [], -1, 0
        if not extra:
            if d == 0:
                paths.append([-1] * A), lens.append(0), drawn.append(-1)
                continue
            path, node, start = [0], 0, 1
        left, total = row(target, node), Fraction(1)
        for t in range(start, d):
            if len(path) == A:
                break
            if par[t] != node or (node == -1 and not extra):
                continue
            tok = int(tokens[b, t])
            if not 0 <= tok < V:
                continue
            q = row(draft, node) if draft is not None else [Fraction(int(x == tok)) for x in range(V)]
            # (uniforms are compared as given: 1 or more accepts nothing that q covers)
            if u[t] is not None and Fraction(float(uniforms[b, t])) * q[tok] < left[tok] / total:
                path.append(t)
                node = t
                left, total = row(target, node), Fraction(1)
                continue
            rest = [max(x - total * y, Fraction(0)) for x, y in zip(left, q)] if draft is not None else \
                [Fraction(0) if x == tok else y for x, y in enumerate(left)]
            if sum(rest) > 0:
                left, total = rest, sum(rest)
        z = sum(left)
        token = -1
        if z > 0:
            run = Fraction(0)
            want = (u[T] if u[T] is not None else 0) * z
            for x, y in enumerate(left):
                run += y
                if y > 0 and (run > want or run == z):
                    token = x
                    break
        paths.append(path + [-1] * (A - len(path)))
        lens.append(len(path))
        drawn.append(token)
    return paths, lens, drawn


def paged_prefill(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens, scale, causal=True, window_left=-1, k_scale=1.0,
                  v_scale=1.0):
    """(out, lse, absv, reach) for every packed row, as spec.tree_attention gives
    them; rows of no request stay NaN."""
    N, Hq, D = q.shape
    ps, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    Q, bt = _f64(q), block_table.cpu().numpy()
    out, absv = np.full((N, Hq, D), np.nan), np.zeros((N, Hq, D))
    lse, reach = np.full((N, Hq), np.nan), np.zeros((N, Hq))
    cu = cu_seqlens_q.tolist()
    for b in range(len(cu) - 1):
        d, n = cu[b + 1] - cu[b], max(0, min(int(seq_lens[b]), bt.shape[1] * ps))
        if d <= 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        t = np.arange(d)
        hi = n - d + t + 1 if causal else np.full(d, n)
        lo = np.zeros(d, dtype=np.int64) if window_left < 0 else np.maximum(0, n - d + t - window_left)
        key = np.arange(n)
        seen = (key[None] < hi[:, None]) & (key[None] >= lo[:, None])
        some = seen.any(1)
        out[rows], lse[rows] = 0.0, -np.inf
        if not some.any():
            continue
        first = int(lo[some].min())                        # earlier pages may be gone
        pages = np.zeros(-(-n // ps), dtype=np.int64)
        pages[first // ps:] = bt[b, first // ps:-(-n // ps)]
        used = key[first:]
        K, V = (c.float().view(-1, Hkv, D)[torch.from_numpy(pages[used // ps] * ps + used % ps)] for c in (k_cache, v_cache))
        K, V = _f64(K) * k_scale, _f64(V) * v_scale
        seen = seen[:, first:]
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            # Keys that no row sees may be NaN.
            ok = seen.any(0)
            k, v = np.where(ok[:, None], k, 0.0), np.where(ok[:, None], v, 0.0)
            x = Q[rows, h]
            s = np.where(seen, x @ k.T * scale, -np.inf)
            m = np.where(some, s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - m[:, None])
            z = np.where(some, e.sum(1), 1.0)
            out[rows, h] = e @ v / z[:, None]
            absv[rows, h] = e @ np.abs(v) / z[:, None]
            lse[rows, h] = np.where(some, m + np.log(z), -np.inf)
            reach[rows, h] = np.where(seen, np.abs(x) @ np.abs(k).T, 0.0).max(1) * abs(scale)
    return out, lse, absv, reach
