"""The paged cache's calls in NumPy float64, one sequence and head at a time.

A cache is (k, v [n_pages, Hkv, page, d], table [B, max_pages]); slot s of
sequence b is row s % page of page table[b, s // page].  A page outside the
pool stands for slots that the call leaves out.
"""

import math

import numpy as np


def places(table_row, n, page_size, n_pages):
    """(page, row, valid) of slots 0 .. n-1."""
    s = np.arange(n)
    page = np.asarray(table_row, dtype=np.int64)[s // page_size]
    return page, s % page_size, (page >= 0) & (page < n_pages)


def decode(q, k, v, table, n_slots, scale):
    """q [B, Hq, d] -> o [B, Hq, d], lse [B, Hq], p {(b, h): (page, row, weights
    summed over the G heads)}, and per (b, head) the sums the error bounds
    need: largest sum_e |q_e k_e| * scale over the slots, and sum_s p_s |v_s|."""
    B, Hq, d = q.shape
    n_pages, Hkv, ps, _ = k.shape
    G = Hq // Hkv
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -math.inf)
    reach, spread = np.zeros((B, Hq)), np.zeros((B, Hq, d))
    weights = {}
    for b in range(B):
        page, row, ok = places(table[b], int(n_slots[b]), ps, n_pages)
        page, row = page[ok], row[ok]
        for h in range(Hkv):
            kk, vv = k[page, h, row], v[page, h, row]
            total = np.zeros(len(page))
            for g in range(h * G, (h + 1) * G):
                if len(page) == 0:
                    continue
                s = (kk @ q[b, g]) * scale
                top = s.max()
                p = np.exp(s - top)
                lse[b, g] = top + math.log(p.sum())
                p /= p.sum()
                o[b, g] = p @ vv
                total += p
                reach[b, g] = (np.abs(kk) @ np.abs(q[b, g])).max() * scale
                spread[b, g] = p @ np.abs(vv)
            weights[b, h] = (page, row, total)
    return o, lse, weights, reach, spread


def rope(x, pos, base):
    """Rotate-half RoPE of x [..., d] at position pos."""
    half = x.shape[-1] // 2
    if not base > 1.0:
        return x.copy()
    ang = pos * base ** (-2.0 * np.arange(half) / x.shape[-1])
    c, s = np.cos(ang), np.sin(ang)
    x1, x2 = x[..., :half], x[..., half:]
    return np.concatenate([x1 * c - x2 * s, x2 * c + x1 * s], -1)


def evict(k, v, weight, slot_pos, table, n_slots, pos, keep, sinks, recent):
    """Cuts in place; returns {(b, h): (movers, holes)}."""
    n_pages, Hkv, ps, _ = k.shape
    moved = {}
    for b in range(table.shape[0]):
        n = int(n_slots[b])
        if n <= keep:
            continue
        page, row, ok = places(table[b], n, ps, n_pages)
        if not ok.all():
            continue
        for h in range(Hkv):
            w = weight[page, h, row].astype(np.float64)
            p = slot_pos[page, h, row].astype(np.int64)

            def rank(s):
                held = p[s] < sinks or p[s] > int(pos[b]) - recent
                if held:
                    return (0, 0.0, s)
                return (2, 0.0, s) if math.isnan(w[s]) else (1, -w[s], s)

            order = sorted(range(n), key=rank)
            kept, dropped = sorted(order[:keep]), sorted(order[keep:])
            movers = [s for s in kept if s >= keep]
            holes = [s for s in dropped if s < keep]
            assert len(movers) == len(holes)
            for x in (k, v, weight, slot_pos):
                x[page[holes], h, row[holes]] = x[page[movers], h, row[movers]]
            moved[b, h] = (movers, holes)
    return moved
