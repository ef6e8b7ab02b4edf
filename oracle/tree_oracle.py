"""64-bit CPU forms of the operators of a step of trees (test infrastructure).

Plain restatements of the definitions in include/csa2.h, node by node; they
share no code with the CUDA library.  Formats and the rotation come from
csa2_oracle.
"""
from __future__ import annotations

import numpy as np

from oracle import csa2_oracle as O
from oracle import paged_oracle as PO


def head_norm(x, weight, eps):
    """Rows x [..., 512] normed (weight None: as they are)."""
    return x if weight is None else PO.rmsnorm(x.reshape(-1, x.shape[-1]), weight, eps).reshape(x.shape)


def turned(x, pos, theta=10000.0):
    """Rows x [n][..., 512] turned by their tokens' positions."""
    flat = x.reshape(len(pos), -1, x.shape[-1])
    rows = [O.rope(flat[i], np.full(flat.shape[1], p), theta) for i, p in enumerate(pos)]
    return np.stack(rows).reshape(x.shape) if len(pos) else x


def lines(parent, q_start, r):
    """Of request r's nodes the way down to each, itself at the end; None where a parent is none."""
    a, b = int(q_start[r]), int(q_start[r + 1])
    out = []
    for i in range(b - a):
        p = int(parent[a + i])
        if p < -1 or p >= i or (p >= 0 and out[p] is None):
            out.append(None)
        else:
            out.append((out[p] if p >= 0 else []) + [i])
    return out


def tree_plan(parent, q_start, kv_len, window, words, pos, mask):
    """(pos, mask) with the requests' nodes filled in."""
    pos, mask = pos.copy(), mask.copy()
    for r in range(len(kv_len)):
        a, n = int(q_start[r]), int(q_start[r + 1]) - int(q_start[r])
        good = kv_len[r] >= n
        for i, line in enumerate(lines(parent, q_start, r)):
            row = np.zeros(words, np.uint64)
            pos[a + i] = -1
            if line is not None and good:
                pos[a + i] = int(kv_len[r]) - n + len(line) - 1
                for j in line[-window:] if window else line:
                    row[j // 32] |= np.uint64(1 << (j % 32))
            mask[a + i] = row.astype(np.uint32).view(np.int32)
    return pos, mask


def tree_attention(q, parent, q_start, kv_len, codes, scales, table, page, window, sm_scale, bad_page=None):
    """(out, lse, (dot, big)) as paged_oracle.paged_attention's, of trees."""
    T, H, D = q.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    dot, big = np.zeros((T, H)), np.zeros((T, H))
    for r in range(len(kv_len)):
        a, n, L = int(q_start[r]), int(q_start[r + 1]) - int(q_start[r]), int(kv_len[r])
        if L < n:
            continue
        p = np.arange(L)
        ids = table[r, p // page] if L else p
        ok = np.array([bad_page is None or not bad_page(int(i)) for i in ids], dtype=bool)
        rows = np.where(ok, ids, 0).astype(np.int64) * page + p % page
        c = PO.latent_rows(codes[rows], None if scales is None else scales[rows]) if L else np.zeros((0, D))
        first = L - n
        for i, line in enumerate(lines(parent, q_start, r)):
            if line is None:
                continue
            see = np.zeros(L, dtype=bool)
            see[max(0, first + len(line) - window) if window else 0:first] = True
            see[[first + j for j in (line[-window:] if window else line)]] = True
            seen = np.flatnonzero(see & ok)
            if not len(seen):
                continue
            x = sm_scale * (q[a + i].astype(np.float64) @ c[seen].T)
            dot[a + i] = np.max(np.abs(q[a + i]).astype(np.float64) @ np.abs(c[seen]).T, axis=1)
            big[a + i] = np.max(np.abs(c[seen]))
            m = x.max(axis=1, keepdims=True)
            e = np.exp(x - m)
            s = e.sum(axis=1, keepdims=True)
            out[a + i] = (e / s) @ c[seen]
            lse[a + i] = (m + np.log(s))[:, 0]
    return out, lse, (dot, big)


def token_logprobs(x, scale, tokens, top):
    """(logprobs, lse, entropy, ids, best) of fp64 rows x."""
    n, V = x.shape
    given = tokens.shape[1]
    logprobs, lse, entropy = np.full((n, given), -np.inf), np.full(n, -np.inf), np.zeros(n)
    ids, best = np.full((n, top), -1, np.int32), np.full((n, top), -np.inf)
    for r in range(n):
        if np.isnan(x[r]).any() or np.isposinf(x[r]).any():
            logprobs[r], lse[r], entropy[r], best[r] = np.nan, np.nan, np.nan, np.nan
            continue
        m = x[r].max()
        if np.isneginf(m):
            continue
        y = (x[r] - m) * scale
        e = np.exp(y)
        s = e.sum()
        lse[r] = m * scale + np.log(s)
        entropy[r] = np.log(s) - (e * np.where(e > 0, y, 0.0)).sum() / s
        for i, t in enumerate(tokens[r]):
            if 0 <= t < V:
                logprobs[r, i] = y[t] - np.log(s)
        order = np.lexsort((np.arange(V), -x[r]))[:top]
        order = order[x[r][order] > -np.inf]
        ids[r, :len(order)], best[r, :len(order)] = order, y[order] - np.log(s)
    return logprobs, lse, entropy, ids, best


def tree_commit(parent, token, choice, q_start, kv_len, page, planes, table, free, n_free, n_pages, cached, n_tokens, bad=()):
    """(path, accepted, next, cached, free, n_free, planes) after a step; the requests of `bad` are those whose bounds do not
    hold, which keep nothing (kv_len, q_start otherwise good)."""
    R = len(kv_len)
    path, accepted, nxt = np.full(n_tokens, -1, np.int32), np.zeros(R, np.int32), np.full(R, -1, np.int64)
    cached, free, planes = cached.copy(), free.copy(), [p.copy() for p in planes]
    back = []
    for r in range(R):
        a, n, L = int(q_start[r]), int(q_start[r + 1]) - int(q_start[r]), int(kv_len[r])
        if n == 0 or r in bad:
            continue
        way = []
        if parent[a] == -1:
            way = [0]
            while True:
                on = [i for i in range(way[-1] + 1, n) if parent[a + i] == way[-1] and token[a + i] == choice[a + way[-1]]]
                if not on:
                    break
                way.append(on[0])
        path[a:a + len(way)] = way
        accepted[r] = len(way)
        nxt[r] = choice[a + way[-1]] if way else -1
        first = L - n
        row = lambda p: int(table[r, p // page]) * page + p % page  # noqa: E731
        held = [[p[row(first + j)].copy() for p in planes] for j in way]
        for j, rows in enumerate(held):
            for p, v in zip(planes, rows):
                p[row(first + j)] = v
        cached[r] = first + len(way)
        back += [int(i) for i in table[r, -(-int(cached[r]) // page):-(-L // page)]]
    for i, page_id in enumerate(reversed(back)):
        free[n_free + i] = page_id
    return path, accepted, nxt, cached, free, n_free + len(back), planes
