"""Float64 oracle of the prompt and page operators (numpy, no shared code with
the GPU path): chunk attention over a paged cache, forking and compacting.
"""
from __future__ import annotations

import numpy as np


def append(pool, new, page_table, kv_len, q_start):
    """pool with the new rows of every request at their positions (a page id
    outside the pool takes none)."""
    pool = pool.copy()
    P = pool.shape[1]
    for b, kv in enumerate(kv_len):
        for i, t in enumerate(range(q_start[b], q_start[b + 1])):
            page = page_table[b][(kv + i) // P]
            if 0 <= page < pool.shape[0]:
                pool[page, (kv + i) % P] = new[t]
    return pool


def rows_of(pool, table_row, n):
    """The first n cached rows of a request, in position order (zeros on a
    page id outside the pool)."""
    P = pool.shape[1]
    out = np.zeros((n,) + pool.shape[2:], dtype=np.float64)
    for j in range(-(-n // P)):
        page = table_row[j]
        if 0 <= page < pool.shape[0]:
            m = min(P, n - j * P)
            out[j * P:j * P + m] = pool[page, :m]
    return out


def chunk_attention(q, k_pool, v_pool, page_table, kv_len, q_start, scale):
    """Attention of the new rows over pools that already hold them.  Returns
    (out, weight, reach): the result [T, Hq, D] (NaN where no request has the
    row), sum_j w_j |v_j|, and per row the largest sum_d |q_d k_d| * scale (what
    rounding errors scale with)."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    out = np.full((T, Hq, D), np.nan)
    weight = np.full((T, Hq, D), np.nan)
    reach = np.zeros((T, Hq, 1))
    q = q.astype(np.float64)
    for b, kv in enumerate(kv_len):
        n = q_start[b + 1] - q_start[b]
        if n == 0:
            continue
        k = rows_of(k_pool, page_table[b], kv + n)
        v = rows_of(v_pool, page_table[b], kv + n)
        for i, t in enumerate(range(q_start[b], q_start[b + 1])):
            seen = kv + i + 1
            for g in range(Hkv):
                kk, vv, qq = k[:seen, g], v[:seen, g], q[t, g * G:(g + 1) * G]
                s = qq @ kk.T * scale
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                out[t, g * G:(g + 1) * G] = w @ vv
                weight[t, g * G:(g + 1) * G] = w @ np.abs(vv)
                reach[t, g * G:(g + 1) * G, 0] = (np.abs(qq) @ np.abs(kk).T).max(-1) * scale
    return out, weight, reach


def fork(parent, reserve, kv_len, pages_used, page_table, next_free, num_pages, P):
    """(next_kv_len, next_pages_used, next_table, next_free, copies): copies is
    a list of (old page, new page, rows)."""
    cols = len(page_table[0])
    seen, copies, full = set(), [], False
    # a parent's first slot is its first one in the list, whether or not it can be made
    first = {}
    for r, p in enumerate(parent):
        first.setdefault(p, r)
    want_free = next_free
    lens, counts, rows = [], [], []
    for r, p in enumerate(parent):
        row, kv = [], 0
        if 0 <= p < len(kv_len):
            kv, more, used = kv_len[p], reserve[r], pages_used[p]
            need = -(-(kv + more) // P)
            ok = kv >= 0 and more >= 0 and -(-kv // P) <= used <= cols and need <= cols
            if ok:
                have = used if first[p] == r else kv // P
                need = max(need, used if first[p] == r else -(-kv // P))
                if need > have and want_free + need - have > num_pages:
                    full = True
                if need > have and full:
                    kv = 0
                else:
                    row = list(page_table[p][:have]) + list(range(want_free, want_free + need - have))
                    if first[p] != r and kv % P:
                        copies.append((page_table[p][have], want_free, kv % P))
                    want_free += need - have
            else:
                kv = 0
        lens.append(kv)
        counts.append(len(row))
        rows.append(row + [-1] * (cols - len(row)))
    return lens, counts, rows, want_free, copies


def compact(pages_used, page_table, num_pages):
    """(next_table, next_free, moves): moves is a list of (old, new) pages."""
    cols = len(page_table[0])
    cut = [min(max(u, 0), cols) for u in pages_used]
    live = {p for row, u in zip(page_table, cut) for p in row[:u] if 0 <= p < num_pages}
    L = len(live)
    moves = list(zip(sorted(p for p in live if p >= L), sorted(set(range(L)) - live)))
    to = dict(moves)
    rows = [[to.get(p, p) for p in row[:u]] + [-1] * (cols - u) for row, u in zip(page_table, cut)]
    return rows, L, moves
