"""64-bit CPU forms of the paged-cache operators (test infrastructure).

Plain restatements of the definitions in include/csa2.h, request by request
and row by row; they share no code with the CUDA library.  Formats come from
csa2_oracle (E2M1, E4M3).
"""
from __future__ import annotations

import numpy as np

from oracle import csa2_oracle as O


def page_plan(cached, added, page, table, free, n_free, n_pages, max_new):
    """(table, q_start, kv_len, slots, pos, n_free, served) of one step."""
    R, max_pages = len(cached), table.shape[1]
    table = table.copy()
    slots, pos = np.full(max_new, -1, np.int64), np.full(max_new, -1, np.int64)
    q_start, kv_len = np.zeros(R + 1, np.int32), np.zeros(R, np.int32)
    pages = lambda n: -(-int(n) // page)  # noqa: E731
    served = all(c >= 0 and a >= 0 and int(c) + int(a) <= max_pages * page for c, a in zip(cached, added))
    if served:
        need = sum(pages(int(c) + int(a)) - pages(c) for c, a in zip(cached, added))
        served = sum(int(a) for a in added) <= max_new and 0 <= n_free <= n_pages and need <= n_free
    if not served:
        return table, q_start, kv_len, slots, pos, n_free, False
    at = 0
    for r in range(R):
        c, a = int(cached[r]), int(added[r])
        for j in range(pages(c), pages(c + a)):
            n_free -= 1
            table[r, j] = free[n_free] if 0 <= free[n_free] < n_pages else -1
        for p in range(c, c + a):
            page_id = int(table[r, p // page])
            slots[at] = page_id * page + p % page if 0 <= page_id < n_pages else -1
            pos[at] = p
            at += 1
        q_start[r + 1], kv_len[r] = at, c + a
    return table, q_start, kv_len, slots, pos, n_free, True


def latent_rows(codes, scales):
    """float64 latents of FP4 rows (codes, scales) or of E4M3 rows (scales None)."""
    if scales is None:
        return O.e4m3_decode(codes)
    return O.dequantize_fp4(O.unpack_codes(codes), scales)


def paged_attention(q, q_start, kv_len, codes, scales, table, page, window, sm_scale, bad_page=None):
    """(out, lse, reach) per token and head over the tokens that q_start covers.  reach: per token and head the
    largest sum over channels of |q||c| and the largest |c| that the row sees, for error bounds.  `bad_page`(id):
    pages that no one sees."""
    T, H, D = q.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    dot, big = np.zeros((T, H)), np.zeros((T, H))
    for r in range(len(kv_len)):
        a, b, L = int(q_start[r]), int(q_start[r + 1]), int(kv_len[r])
        p = np.arange(L)
        ids = table[r, p // page] if L else p
        ok = np.array([bad_page is None or not bad_page(int(i)) for i in ids], dtype=bool)
        rows = np.where(ok, ids, 0).astype(np.int64) * page + p % page
        c = latent_rows(codes[rows], None if scales is None else scales[rows]) if L else np.zeros((0, D))
        for i in range(b - a):
            t = L - (b - a) + i
            seen = np.flatnonzero((p <= t) & ok & ((p > t - window) if window else True))
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


def rmsnorm(h, weight, eps):
    """fp64 y of rows h (already bf16 values)."""
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * weight


def matvec(x, x_scales, codes, scales, alpha):
    """(out, reach): alpha x W^T and the sum of |x||W| of each value."""
    w = O.dequantize_fp4(O.unpack_codes(codes), scales)
    x = x if x_scales is None else x * x_scales[:, None].astype(np.float64)
    return alpha * (x @ w.T), abs(alpha) * (np.abs(x) @ np.abs(w).T)
