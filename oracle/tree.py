"""64-bit oracle of the operators of a step with drafted trees (numpy, plain loops),
written from their definitions: it shares no code with the CUDA library or its
binding.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .serving import gather


def ancestors(parents, i):
    """Node i and everything above it; a parent that does not lie in front of its node ends the chain."""
    chain = [i]
    while 0 <= parents[chain[-1]] < chain[-1]:
        chain.append(int(parents[chain[-1]]))
    return chain


def attn_tree(q, k_cache, v_cache, page_table, kv_lens, q_offsets, parents, scale=None):
    """(out, lse, size, score) as oracle.serving.attn_paged returns them."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    G = Hq // k_cache.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, score = np.full((Hq, T), -np.inf), np.zeros((T, Hq))
    for r in range(len(kv_lens)):
        q0, q1, L = int(q_offsets[r]), int(q_offsets[r + 1]), int(kv_lens[r])
        base = L - (q1 - q0)
        k, v = (gather(c, page_table, r, L) for c in (k_cache, v_cache))
        for i in range(q1 - q0):
            at = list(range(max(base, 0))) + sorted(base + j for j in ancestors(parents[q0:q1], i) if base + j >= 0)
            if not at:
                continue
            for h in range(Hq):
                kk, vv = k[at, h // G], v[at, h // G]
                x = kk @ q[q0 + i, h] * scale
                score[q0 + i, h] = (np.abs(kk) @ np.abs(q[q0 + i, h])).max() * abs(scale)
                p = np.exp(x - x.max())
                out[q0 + i, h] = p @ vv / p.sum()
                size[q0 + i, h] = p @ np.abs(vv) / p.sum()
                lse[h, q0 + i] = x.max() + np.log(p.sum())
    return out, lse, size, score


def distribution(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Weights of one row's tokens, those that are not kept 0 (all 0: no choice)."""
    x = np.asarray(logits, np.float64).copy()
    w = np.zeros(len(x))
    x[~(x >= -2.0 ** 126)] = -np.inf
    x = np.minimum(x, 2.0 ** 126)
    if not temperature >= 0 or math.isinf(temperature) or not np.isfinite(x).any():
        return w
    order = sorted((i for i in range(len(x)) if np.isfinite(x[i])), key=lambda i: (-x[i], i))
    if temperature == 0:
        w[order[0]] = 1.0
        return w
    if 0 < top_k < len(x):
        order = order[:top_k]
    e = np.array([math.exp((x[i] - x[order[0]]) / max(temperature, 2.0 ** -100)) for i in order])
    if top_p < 1:
        whole, run, end = math.fsum(e), 0.0, 0
        while end < len(order):
            run += e[end]
            end += 1
            if abs(run - top_p * whole) > 1e-9 * whole:
                if run > top_p * whole:
                    break
            else:  # too near for sums in 64 bits; a weight that 64 bits hold as 0 is above 0
                exact = sum(map(Fraction, e[:end])) - Fraction(top_p) * sum(map(Fraction, e))
                if exact > 0 or (exact == 0 and e[-1] > 0):
                    break
        order, e = order[:end], e[:end]
    for i, y in zip(order, e):
        if not min_p > 0 or y >= min(min_p, 1.0):
            w[i] = y
    return w


def sample(weights, u):
    """The first token whose running sum exceeds u times the whole; 0 where there is no weight."""
    c = np.cumsum(weights)
    z = int(np.searchsorted(c, float(u) * c[-1], side="right"))
    return z if z < len(c) else 0


def accept(sampled, tokens, parents, q_offsets, max_path):
    """(path, out_tokens, num_accepted) of the walks."""
    R = len(q_offsets) - 1
    path, out, count = np.full((R, max_path), -1, np.int32), np.full((R, max_path), -1, np.int32), np.zeros(R, np.int32)
    for r in range(R):
        q0, q1 = int(q_offsets[r]), int(q_offsets[r + 1])
        at = 0 if q1 > q0 else None
        while at is not None and count[r] < max_path:
            path[r, count[r]], out[r, count[r]] = at, sampled[q0 + at]
            count[r] += 1
            at = next((j for j in range(at + 1, q1 - q0)
                       if parents[q0 + j] == at and tokens[q0 + j] == sampled[q0 + at]), None)
    return path, out, count


def compact(cache, page_table, kv_lens, q_offsets, path, count):
    """(cache [..., pages, page_size, H, D] after the move, new lengths)."""
    cache, P = cache.copy(), cache.shape[-3]
    new = []
    for r in range(len(kv_lens)):
        base = int(kv_lens[r]) - int(q_offsets[r + 1] - q_offsets[r])
        at = [(page_table[r][(base + int(k)) // P], (base + int(k)) % P) for k in path[r][:count[r]]]
        rows = [cache[..., g, i, :, :].copy() for g, i in at]
        for j, x in enumerate(rows):
            cache[..., page_table[r][(base + j) // P], (base + j) % P, :, :] = x
        new.append(base + int(count[r]))
    return cache, new


def _take(refs):
    for g in range(len(refs)):
        if refs[g] == 0:
            refs[g] = 1
            return g
    return -1


def resize(page_table, old, new, refs, P):
    """(page_table, refs, missing)."""
    table, refs, missing = [list(map(int, r)) for r in page_table], list(map(int, refs)), 0
    pages = lambda n: -(-int(n) // P)  # noqa: E731
    for r, (a, b) in enumerate(zip(old, new)):
        for j in range(pages(b), pages(a)):
            if table[r][j] != -1:
                refs[table[r][j]] -= 1
            table[r][j] = -1
    for r, (a, b) in enumerate(zip(old, new)):
        for j in range(pages(a), pages(b)):
            table[r][j] = _take(refs)
            missing += table[r][j] < 0
    return np.array(table), np.array(refs), missing


def fork(page_table, lens, src, dst, refs, P):
    """(page_table, lens, refs, copy_src, copy_dst, copy_rows, missing)."""
    table, refs, lens = [list(map(int, r)) for r in page_table], list(map(int, refs)), list(map(int, lens))
    out, missing = [], 0
    for a, b in zip(src, dst):
        full, rest = divmod(lens[a], P)
        for j in range(full):
            table[b][j] = table[a][j]
            refs[table[a][j]] += 1
    for a, b in zip(src, dst):
        full, rest = divmod(lens[a], P)
        lens[b] = lens[a]
        if rest:
            table[b][full] = _take(refs)
            missing += table[b][full] < 0
        out.append((table[a][full] if rest else -1, table[b][full] if rest else -1, rest))
    s, d, n = zip(*out) if out else ((), (), ())
    return np.array(table), np.array(lens), np.array(refs), list(s), list(d), list(n), missing
