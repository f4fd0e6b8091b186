"""fp64 oracle of the cache operators: attention weights, eviction and the 4-bit cache.

Plain numpy, written from the operators' definitions; shares no code with the
package.  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------------------
# attention and its weights

def attend(q, k, v, scale, heads_per_kv):
    """One row: q [H_q][D], k and v [H_kv][N][D], all float64.  Returns out [H_q][D], the weights summed over each
    KV head's query heads [H_kv][N], sum_t w |v| [H_q][D], and sum_d |q k| [H_q] at its largest (for tolerances)."""
    H_q, D = q.shape
    H_kv, N, _ = k.shape
    out, reach = np.zeros((H_q, D)), np.zeros((H_q, D))
    weights, size = np.zeros((H_kv, N)), np.zeros(H_q)
    if N == 0:
        return out, weights, reach, size
    for hq in range(H_q):
        h = hq // heads_per_kv
        x = scale * (k[h] @ q[hq])
        with np.errstate(invalid="ignore"):
            w = np.exp(x - np.nanmax(x)) if not np.isnan(x).all() else x
        w = w / w.sum()
        out[hq] = w @ v[h]
        reach[hq] = w @ np.abs(v[h])
        size[hq] = np.nanmax(np.abs(k[h]) @ np.abs(q[hq])) if not np.isnan(x).all() else 0.0
        weights[h] += w
    return out, weights, reach, size


# ---------------------------------------------------------------------------
# eviction

def evict_source(scores, n, budget, recent):
    """Where each of the `budget` slots' tokens come from after an eviction of one (row, KV head) with n > budget
    tokens and scores [>= n]."""
    first, older = budget - recent, n - recent
    key = [(-np.inf if np.isnan(s) else float(s)) for s in scores[:older]]
    ranked = sorted(range(older), key=lambda t: (-key[t], t))
    kept = sorted(ranked[:first])
    stay = set(t for t in kept if t < first)
    movers = [t for t in kept if t >= first]
    source = []
    for slot in range(first):
        source.append(slot if slot in stay else movers.pop(0))
    assert not movers
    return source + list(range(older, n))


def evict(scores, positions, planes, block_table, lens, budget, recent):
    """New (scores, positions, planes, lens): arrays [B][H][T], [B][H][T], list of [pages][H][16][X], [B]."""
    scores, positions, planes = scores.copy(), positions.copy(), [p.copy() for p in planes]
    B, H, _ = scores.shape
    new_lens = [min(n, budget) for n in lens]
    for i in range(B):
        n = lens[i]
        if n <= budget:
            continue
        for h in range(H):
            src = evict_source(scores[i, h], n, budget, recent)
            old_s, old_p = scores[i, h].copy(), positions[i, h].copy()
            scores[i, h, :budget], positions[i, h, :budget] = old_s[src], old_p[src]
            scores[i, h, budget:n] = 0.0
            for plane in planes:
                rows = np.stack([plane[block_table[i, t // PAGE], h, t % PAGE].copy() for t in src]) if src else []
                for slot in range(budget):
                    plane[block_table[i, slot // PAGE], h, slot % PAGE] = rows[slot]
    return scores, positions, planes, new_lens


# ---------------------------------------------------------------------------
# the 4-bit cache

def quantise(x):
    """float64 [..., D] -> (codes [..., D], scale bytes [..., D/32]) by nearest value, ties to the even code."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(blocks).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(blocks), blocks, 0.0)).max(-1))
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))), 0)
    scale = np.where(amax > 0, np.clip(e + 125, 1, 254), 0).astype(int)
    step = 2.0 ** (scale.astype(float) - 127)
    y = np.where(bad[..., None], 0.0, np.abs(np.where(np.isfinite(blocks), blocks, 0.0)) / step[..., None])
    far = np.abs(y[..., None] - GRID)
    near = far == far.min(-1, keepdims=True)
    code = np.argmin(np.where(near, np.arange(8) % 2, 2), -1)  # of equally near codes the even one
    code = np.where(np.signbit(blocks) & ~bad[..., None], code | 8, code)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape), np.where(bad, 255, scale)


def values(code, scale):
    """float64 values of codes [..., D] under scale bytes [..., D/32]."""
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(float) - 127))
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    return (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)


def code_bytes(D, is_v):
    """(byte, shift) of every dim's code in a token's row."""
    byte, shift = [], []
    for d in range(D):
        b, rest = divmod(d, 32)
        if is_v:
            r, j = divmod(rest, 4)
            byte.append(r * D // 16 + 2 * b + j // 2)
        else:
            c, j = divmod(rest, 8)
            byte.append(c * D // 8 + 4 * b + j // 2)
        shift.append(4 * (j % 2))
    return np.array(byte), np.array(shift)


def put(record, slot, D, is_v, code, scale):
    """Write one token's codes and scale bytes into a record (uint8 [17 D]), in place."""
    byte, shift = code_bytes(D, is_v)
    row = record[(8 * D if is_v else 0) + slot * (D // 2):][:D // 2]
    row[:] = 0
    np.bitwise_or.at(row, byte, (code << shift).astype(np.uint8))
    at = 16 * D + (D // 2 if is_v else 0) + slot * (D // 32)
    record[at:at + D // 32] = scale


def get(record, D, is_v):
    """(codes [16][D], scale bytes [16][D/32]) of a record."""
    byte, shift = code_bytes(D, is_v)
    rows = record[(8 * D if is_v else 0):][:8 * D].reshape(16, D // 2)
    at = 16 * D + (D // 2 if is_v else 0)
    return (rows[:, byte].astype(int) >> shift) & 15, record[at:at + D // 2].reshape(16, D // 32).astype(int)


def row_values(pool, table_row, n, h, is_v):
    """float64 [n][D] of one row's cached K or V for KV head h (pool uint8 [pages][H][17 D])."""
    D = pool.shape[2] // 17
    got = [values(*get(pool[p, h], D, is_v)) for p in table_row[:-(-n // PAGE)]]
    return np.concatenate(got)[:n] if got else np.zeros((0, D))
