"""64-bit oracle of the grouped-query serving operators (numpy, plain loops over
requests and heads), written from their definitions: it shares no code with the
CUDA library or its binding.

Where a rounding bound needs the size of what was added up, the functions return
that too: `size` holds, for every result, the sum of the absolute values of its
terms.
"""
from __future__ import annotations

import numpy as np


def rotation_matrix(cos, sin, D, interleaved):
    """[D, D] matrix of one token's rotation; cos, sin: rot_dim / 2 values each."""
    h = len(cos)
    m = np.eye(D)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        m[a, a], m[a, b], m[b, a], m[b, b] = cos[i], -sin[i], sin[i], cos[i]
    return m


def _matrices(positions, cos_sin, D, interleaved):
    if cos_sin is None:
        return [np.eye(D)] * len(positions)
    h = cos_sin.shape[1] // 2
    t = np.asarray(cos_sin, np.float64)
    return [rotation_matrix(t[p, :h], t[p, h:], D, interleaved) for p in positions]


def norm_rope(x, w, positions, cos_sin, eps, interleaved):
    """(result, size) of the norm and rotation of x [T, H, D]."""
    x = np.asarray(x, np.float64)
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    out, size = np.empty_like(y), np.empty_like(y)
    for t, m in enumerate(_matrices(positions, cos_sin, x.shape[-1], interleaved)):
        out[t], size[t] = y[t] @ m.T, np.abs(y[t]) @ np.abs(m).T
    return out, size


def norm_rope_backward(x, w, positions, cos_sin, eps, interleaved, dout):
    """(dx, size of dx, dw, size of dw) of sum(dout * norm_rope(x)); dw is None without a weight."""
    dout = np.asarray(dout, np.float64)
    g, gs = np.empty_like(dout), np.empty_like(dout)
    for t, m in enumerate(_matrices(positions, cos_sin, dout.shape[-1], interleaved)):
        g[t], gs[t] = dout[t] @ m, np.abs(dout[t]) @ np.abs(m)
    if w is None:
        return g, gs, None, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dx = r * (g * w - xh * (g * w * xh).mean(-1, keepdims=True))
    size = r * (gs * np.abs(w) + np.abs(xh) * (gs * np.abs(w * xh)).mean(-1, keepdims=True))
    return dx, size, (g * xh).sum((0, 1)), (gs * np.abs(xh)).sum((0, 1))


def token_places(q_offsets, kv_lens, page_table, page_size):
    """(request, position, page, row) of every packed token of the batch."""
    out = []
    for r in range(len(kv_lens)):
        n = int(q_offsets[r + 1] - q_offsets[r])
        for i in range(n):
            p = int(kv_lens[r]) - n + i
            out.append((r, p, int(page_table[r][p // page_size]), p % page_size))
    return out


def gather(cache, page_table, r, length):
    """Positions 0 .. length - 1 of request r: [length, H, D] in 64 bits."""
    P = cache.shape[1]
    rows = [np.asarray(cache[page_table[r][p // P], p % P], np.float64) for p in range(length)]
    return np.stack(rows) if rows else np.zeros((0,) + cache.shape[2:])


def attn_paged(q, k_cache, v_cache, page_table, kv_lens, q_offsets, causal, scale=None):
    """(out, lse, size, score): out [T, Hq, D], lse [Hq, T]; size = sum of p |v| of
    every output, score [T, Hq] = largest sum of |q_d k_d| scale among the keys seen."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, score = np.full((Hq, T), -np.inf), np.zeros((T, Hq))
    for r in range(len(kv_lens)):
        q0, q1, L = int(q_offsets[r]), int(q_offsets[r + 1]), int(kv_lens[r])
        k, v = (gather(c, page_table, r, L) for c in (k_cache, v_cache))
        for i in range(q1 - q0):
            seen = L if not causal else min(L, max(0, L - (q1 - q0) + i + 1))
            if seen == 0:
                continue
            for h in range(Hq):
                kk, vv = k[:seen, h // G], v[:seen, h // G]
                x = kk @ q[q0 + i, h] * scale
                score[q0 + i, h] = (np.abs(kk) @ np.abs(q[q0 + i, h])).max() * abs(scale)
                m = x.max()
                p = np.exp(x - m)
                out[q0 + i, h] = p @ vv / p.sum()
                size[q0 + i, h] = p @ np.abs(vv) / p.sum()
                lse[h, q0 + i] = m + np.log(p.sum())
    return out, lse, size, score


def verify(target, draft, tokens, offsets, accept_u, sample_u, max_draft):
    """(out_tokens, num_accepted) of the verification; draft None: the draft took its most likely token."""
    R, V = len(offsets) - 1, target.shape[1]
    out, acc = np.full((R, max_draft + 1), -1, np.int32), np.zeros(R, np.int32)
    target = np.asarray(target, np.float64)
    for r in range(R):
        t0, n = int(offsets[r]), int(offsets[r + 1] - offsets[r])
        a = 0
        while a < n:
            x = int(tokens[t0 + a])
            if not 0 <= x < V:
                break
            qx = 1.0 if draft is None else float(draft[t0 + a, x])
            if not float(accept_u[t0 + a]) * qx < target[t0 + r + a, x]:
                break
            out[r, a] = x
            a += 1
        w = target[t0 + r + a]
        if a < n:
            q = np.zeros(V) if draft is None else np.asarray(draft[t0 + a], np.float64)
            if draft is None and 0 <= int(tokens[t0 + a]) < V:
                q[int(tokens[t0 + a])] = np.inf
            rest = np.maximum(w - q, 0.0)
            w = rest if rest.sum() > 0 else w
        c = np.cumsum(w)
        z = int(np.searchsorted(c, float(sample_u[r]) * c[-1], side="right"))
        out[r, a], acc[r] = (z if z < V else 0), a
    return out, acc
