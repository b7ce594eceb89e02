"""CPU oracle for the key-value cache's operators: fp64 numpy, one step per definition.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Everything is plain float64 (or
integer) arrays: pools [pages][heads][page][dim] hold the values that the stored elements
stand for, tables and lengths are int arrays.  Nothing is rounded to a storage type here.
"""
from __future__ import annotations

import numpy as np


def slots(table_row, page, pages, n):
    """(page number, place) of the first n slots of a row; page -1 where there is none."""
    j = np.arange(n)
    at = np.asarray(table_row)[j // page].astype(np.int64)
    return np.where((at < 0) | (at >= pages), -1, at), j % page


def gather(pool, table_row, head, n):
    """The head's first n rows [n][dim] of a pool and whether each is there."""
    at, place = slots(table_row, pool.shape[2], pool.shape[0], n)
    return pool[np.maximum(at, 0), head, place], at >= 0


def attend(q, k, v, table, lens, scale, acc=None, decay=1.0):
    """q [rows][q_heads][dim] -> (out, acc_out or None)."""
    rows, q_heads, dim = q.shape
    heads = k.shape[1]
    group = q_heads // heads
    out = np.zeros(q.shape)
    acc_out = None if acc is None else np.array(acc, dtype=np.float64)
    for r in range(rows):
        n = int(lens[r])
        for h in range(heads if n > 0 else 0):
            kk, there = gather(k, table[r], h, n)
            vv, _ = gather(v, table[r], h, n)
            kk, vv = kk[there], vv[there]
            weight = np.zeros(n)
            for g in range(h * group, (h + 1) * group):
                with np.errstate(invalid="ignore"):
                    s = (kk * q[r, g]).sum(axis=1) * scale
                    top = s.max() if s.size else -np.inf
                    if top == -np.inf:  # nothing to attend to
                        continue
                    e = np.exp(s - top)
                    p = e / e.sum()
                    out[r, g] = (p[:, None] * vv).sum(axis=0)
                weight[there] += p
            if acc is not None:
                acc_out[r, h, :n] = decay * acc_out[r, h, :n] + weight
    return out, acc_out


def turned(x, position, rope, norm, eps):
    """One token's heads [heads][dim]: divided by their root mean square, then rotated."""
    x = np.asarray(x, dtype=np.float64)
    if norm is not None:
        x = x / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps) * norm
    if rope is not None:
        half = x.shape[1] // 2
        if not 0 <= position < len(rope):
            return np.full(x.shape, np.nan)
        cos, sin = rope[position, :half], rope[position, half:]
        a, b = x[:, :half], x[:, half:]
        x = np.concatenate([a * cos - b * sin, b * cos + a * sin], axis=1)
    return x


def append(k_pool, v_pool, table, lens, cu, positions, k, v, q=None, rope=None, q_norm=None, k_norm=None, eps=0.0,
           pos=None, acc=None):
    """New pools, totals and positions, rotated queries and lengths; inputs are left alone."""
    k_pool, v_pool = np.array(k_pool), np.array(v_pool)
    pos = None if pos is None else np.array(pos)
    acc = None if acc is None else np.array(acc)
    pages, _, page, _ = k_pool.shape
    cap = table.shape[1] * page
    q_out = None if q is None else np.zeros(q.shape)
    lens = np.clip(np.asarray(lens), 0, cap)
    for r in range(len(lens)):
        for t in range(cu[r], cu[r + 1]):
            if q is not None:
                q_out[t] = turned(q[t], positions[t], rope, q_norm, eps)
            slot = int(lens[r]) + t - cu[r]
            if slot >= cap:
                continue
            at = int(table[r][slot // page])
            if not 0 <= at < pages:
                continue
            k_pool[at, :, slot % page] = turned(k[t], positions[t], rope, k_norm, eps)
            v_pool[at, :, slot % page] = v[t]
            if pos is not None:
                pos[r, :, slot] = positions[t]
            if acc is not None:
                acc[r, :, slot] = 0
    return k_pool, v_pool, q_out, pos, acc, lens + np.diff(cu)


def evict(k_pool, v_pool, table, lens, acc, pos, budget, sink, recent, acc_out, pos_out):
    """New pools, totals (into a copy of acc_out), positions (of pos_out) and lengths."""
    k_pool, v_pool, acc_out, pos_out = (np.array(x) for x in (k_pool, v_pool, acc_out, pos_out))
    pages, heads, page, _ = k_pool.shape
    for r in range(len(lens)):
        n = int(lens[r])
        at, place = slots(table[r], page, pages, n)
        for h in range(heads):
            a, p = np.array(acc[r, h, :n]), np.array(pos[r, h, :n])
            if n > budget:
                newest = p.max()
                # protected slots first, whatever their totals
                key = [(0, 0) if (x < sink or x > newest - recent) else (1, np.inf if np.isnan(y) else -y)
                       for x, y in zip(p.tolist(), a.tolist())]
                kept = sorted(sorted(range(n), key=lambda j: (key[j], j))[:budget])
                kept_set = set(kept)
                gaps = [j for j in range(budget) if j not in kept_set]
                for to, of in zip(gaps, [j for j in kept if j >= budget]):
                    a[to], p[to] = a[of], p[of]
                    if at[to] >= 0 and at[of] >= 0:
                        for pool in (k_pool, v_pool):
                            pool[at[to], h, place[to]] = pool[at[of], h, place[of]]
            m = min(n, budget)
            acc_out[r, h, :m], pos_out[r, h, :m] = a[:m], p[:m]
    return k_pool, v_pool, acc_out, pos_out, np.minimum(lens, budget)


def reserve(table, page, pages, lens, want, held, free, count, max_tokens, shared=None, seen=None):
    """One row after the other: (table, free, cu, positions, slots, granted, held, count), inputs left alone."""
    table, free = np.array(table), np.array(free)
    rows, width = table.shape
    cap = width * page
    stack = list(free[:min(max(int(count), 0), len(free))])
    bottom = len(stack)
    lens = [min(max(int(n), 0), cap) for n in lens]
    held = [min(max(int(h), 0), width) for h in held]
    ask, need, given = [], [], []
    for r in range(rows):
        t = max(int(want[r]), 0)
        ask.append(t if lens[r] + t <= cap else 0)
        need.append(-(-(lens[r] + ask[r]) // page))
        if shared is not None:
            need[r] = max(need[r], min(int(shared[r]), held[r]))
        given += list(table[r, need[r]:held[r]])
        held[r] = min(held[r], max(need[r], 0)) if held[r] > need[r] else held[r]
    stack += given[::-1]  # the first one given back on top
    granted, open_ = [0] * rows, True
    for r in range(rows):
        open_ = open_ and need[r] - held[r] <= len(stack) and sum(granted) + ask[r] <= max_tokens
        if open_:
            granted[r] = ask[r]
            while held[r] < need[r]:
                table[r, held[r]] = stack.pop()
                held[r] += 1
    end = min(len(stack), len(free))
    free[bottom:end] = stack[bottom:end]
    cu = np.concatenate([[0], np.cumsum(granted)]).astype(np.int64)
    positions, slots = np.zeros(max_tokens, dtype=np.int64), np.full(max_tokens, -1, dtype=np.int64)
    for r in range(rows):
        for i in range(granted[r]):
            j = lens[r] + i
            at = int(table[r, j // page])
            positions[cu[r] + i] = (lens[r] if seen is None else int(seen[r])) + i
            slots[cu[r] + i] = at * page + j % page if 0 <= at < pages else -1
    return table, free, cu, positions, slots, granted, held, end


def attend_tokens(q, k, v, table, lens, cu, scale):
    """q [tokens][q_heads][dim], token j of the n of a row of length L over its first L - n + 1 + j slots."""
    out = np.zeros(q.shape)
    for r in range(len(lens)):
        for t in range(cu[r], cu[r + 1]):
            n = int(lens[r]) - int(cu[r + 1]) + 1 + t
            out[t] = attend(q[t:t + 1], k, v, table[r:r + 1], [n], scale)[0][0]
    return out
