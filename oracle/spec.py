"""Plain 64-bit definitions of the speculative-decoding operators -- TEST
INFRASTRUCTURE ONLY, like the rest of this package.

Each is a loop over requests, written from the definition in the header of the
C ABI; nothing here shares code with the library.
"""
from __future__ import annotations

import numpy as np
import torch


def _f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def tree_attention(q, k_cache, v_cache, block_table, seq_lens, tree_mask, scale, draft_lens=None, k_scale=1.0,
                   v_scale=1.0):
    """Returns (out, lse, absv, reach, spread): the outputs [B, T, Hq, D], the
    natural log-sum-exp [B, T, Hq], the softmax-weighted mean of |v| per output
    column, per row the largest sum_i |q_i k_i| * scale over its visible keys
    (what the rounding of an FP32 score scales with), and, for 8-bit caches, the
    largest max_i |q_i| * sum_i |k_i| * scale (what a score is off by when every
    query element is off by a fraction of the row's largest; 0 otherwise)."""
    B, T, Hq, D = q.shape
    ps, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    Q, KC, VC = _f64(q), _f64(k_cache), _f64(v_cache)
    bt, n_all, mask = block_table.cpu().numpy(), seq_lens.cpu().numpy(), tree_mask.cpu().numpy()
    d_all = np.full(B, T) if draft_lens is None else draft_lens.cpu().numpy()
    out, absv = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D))
    lse, reach, spread = np.full((B, T, Hq), -np.inf), np.zeros((B, T, Hq)), np.zeros((B, T, Hq))
    kv8 = k_cache.dtype == torch.float8_e4m3fn
    for b in range(B):
        n = int(n_all[b])
        d = max(0, min(int(d_all[b]), T, n))
        if n == 0 or d == 0:
            continue
        pages = bt[b, :-(-n // ps)].astype(np.int64)
        K = KC[pages].reshape(-1, Hkv, D)[:n] * k_scale
        V = VC[pages].reshape(-1, Hkv, D)[:n] * v_scale
        for t in range(d):
            keys = list(range(n - d)) + [n - d + j for j in range(d) if (int(mask[b, t, j // 32]) >> (j % 32)) & 1]
            if not keys:
                continue
            for h in range(Hq):
                k, v = K[keys, h // G], V[keys, h // G]
                s = k @ Q[b, t, h] * scale
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                lse[b, t, h] = m + np.log(z)
                out[b, t, h] = e @ v / z
                absv[b, t, h] = e @ np.abs(v) / z
                reach[b, t, h] = (np.abs(k) @ np.abs(Q[b, t, h])).max() * abs(scale)
                if kv8:
                    spread[b, t, h] = np.abs(Q[b, t, h]).max() * np.abs(k).sum(1).max() * abs(scale)
    return out, lse, absv, reach, spread


def tree_mask(parents, draft_lens=None):
    """(mask words [B, T, W] int32, depths [B, T] int32); a parent outside
    -1 .. t - 1 counts as -1."""
    P = parents.cpu().numpy()
    B, T = P.shape
    W = -(-T // 32)
    words, depths = np.zeros((B, T, W), dtype=np.uint32), np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        d = T if draft_lens is None else max(0, min(T, int(draft_lens[b])))
        for t in range(d):
            u, depth = t, -1
            while u >= 0:
                words[b, t, u // 32] |= np.uint32(1) << np.uint32(u % 32)
                depth += 1
                up = int(P[b, u])
                u = up if -1 <= up < u else -1
            depths[b, t] = depth
    return torch.from_numpy(words.view(np.int32)), torch.from_numpy(depths)


def page_tables(seq_lens, new_lens, held, free_queue, free_range, page_size, block_table, slot_mapping):
    """Walks the requests one by one.  Returns new copies of (block_table,
    slot_mapping, cu_new, held, free_queue, free_range) and the set of status
    codes the step may report (empty: none)."""
    seq, new = seq_lens.tolist(), new_lens.tolist()
    h = held.tolist()
    q = free_queue.tolist()
    head, count = free_range.tolist()
    bt, shape = block_table.clone(), slot_mapping.shape
    F, B, width = len(q), len(seq), bt.shape[1]
    padded = len(shape) == 2
    slots = torch.full((slot_mapping.numel(),), -1, dtype=torch.int32)
    codes = set()
    ok_range = 0 <= head < F and 0 <= count <= F
    if not ok_range:
        codes.add(1)
    start = head if ok_range else 0
    avail, room = (count, F - count) if ok_range else (0, 0)
    asked = given = taken = returned = 0
    tail = []
    cu = [0]
    total = 0
    for b in range(B):
        first = total
        total += max(0, new[b])
        cu.append(min(total, 2 ** 31 - 1))
        good = 0 <= seq[b] <= width * page_size and 0 <= new[b] <= seq[b] and 0 <= h[b] <= width
        if padded and new[b] > shape[1]:
            good = False
        if not good:
            codes.add(1)
            continue
        want = -(-seq[b] // page_size)
        if want > h[b]:
            asked += want - h[b]
            if asked > avail:
                if ok_range:
                    codes.add(3)
                continue
            for lp in range(h[b], want):
                bt[b, lp] = q[(start + taken) % F]
                taken += 1
            h[b] = want
        elif want < h[b]:
            returned += h[b] - want
            if returned > room:
                codes.add(1)
            else:
                tail += bt[b, want:h[b]].tolist()
                given = returned
                h[b] = want
        for j in range(new[b]):
            pos = seq[b] - new[b] + j
            page = int(bt[b, pos // page_size])
            place = b * shape[1] + j if padded else first + j
            if place >= slots.numel():
                codes.add(1)
                continue
            if 0 <= page < (2 ** 31 - 1) // page_size:
                slots[place] = page * page_size + pos % page_size
            else:
                codes.add(1)
    for i, page in enumerate(tail):
        q[(start + count + i) % F] = page
    left = [(head + taken) % F, count - taken + given] if ok_range else [head, count]

    def i32(v):
        return torch.tensor(v, dtype=torch.int32)

    return bt, slots.view(shape), i32(cu), i32(h), i32(q), i32(left), codes


def commit(path, path_lens, base_lens, block_table, caches, num_layers=1):
    """New copies of the caches after the move, and the new lengths."""
    outs = [c.clone() for c in caches]
    P, ps = caches[0].shape[0], caches[0].shape[1]
    layer = P // num_layers
    new = (base_lens + path_lens).clone()
    for b in range(path.shape[0]):
        base = int(base_lens[b])
        for i in range(int(path_lens[b])):
            src, dst = base + int(path[b, i]), base + i
            sp, dp = int(block_table[b, src // ps]), int(block_table[b, dst // ps])
            for l in range(num_layers):
                for c, o in zip(caches, outs):
                    o[l * layer + dp, dst % ps] = c[l * layer + sp, src % ps]
    return outs, new
