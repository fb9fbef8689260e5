"""The paged key/value cache in plain Python and float64: block tables and
slots from the requests' lengths, the write of new tokens into their pages, and
the attention of every request's new tokens over them.

TEST INFRASTRUCTURE ONLY: only ``tests/`` imports it, and it shares nothing
with the CUDA library.  Everything is written per request, token and head, from
the definitions:

  position j of request b is in page table[b][j // ps], at offset j % ps;
  query i of n is at position p = L - n + i and sees key j iff j <= p and (no
  window, or j > p - window, or j < sinks);
  out = sum_j p_j v_j, p = softmax of scale * q . k_j over the seen keys; 0
  where none is seen.
"""
import numpy as np


def tables(cached, fresh, free_pages, table, page_size, num_pages, rows):
    """-> (table, cu_fresh, kv_len, slots, taken); lengths that fit, or -1 where
    a page is missing."""
    table = np.array(table)
    width = table.shape[1]
    cap = width * page_size
    cu, kv_len, slots, at = [0], [], [-1] * rows, 0
    for b, (c, n) in enumerate(zip(cached, fresh)):
        c, n = max(int(c), 0), max(int(n), 0)
        kv_len.append(min(c + n, cap))
        for j in range(-(-min(c, cap) // page_size), -(-min(c + n, cap) // page_size)):
            page = int(free_pages[at]) if at < len(free_pages) else -1
            table[b, j] = page if 0 <= page < num_pages else -1
            at += 1
        for i in range(n):
            t, j = cu[-1] + i, (c + i) // page_size
            if t < rows and j < width and 0 <= table[b, j] < num_pages:
                slots[t] = int(table[b, j]) * page_size + (c + i) % page_size
        cu.append(cu[-1] + n)
    return table, np.array(cu), np.array(kv_len), np.array(slots, dtype=np.int64), at


def seen(L, n, i, window, sinks):
    """The keys that query i of n sees, of L, as an index array."""
    p = L - n + i
    j = np.arange(max(0, min(L, p + 1)))
    if window > 0:
        j = j[(j > p - window) | (j < sinks)]
    return j


def gather(cache, table_row, L, page_size, num_pages):
    """[L, H_kv, D] of a request's keys (or values), and which have a page."""
    pages = np.array([int(table_row[j // page_size]) for j in range(L)], dtype=np.int64)
    ok = (pages >= 0) & (pages < num_pages)
    off = np.arange(L) % page_size
    return cache[np.where(ok, pages, 0), :, off], ok


def attention(q, k_cache, v_cache, table, cu, kv_len, window, sinks, scale):
    """float64 arrays -> (out [T, H_q, D], sum_j p_j |v_j|, sum |q||k| scale of
    the seen key where it is largest [T, H_q], seen keys [T]); rows of no
    request are NaN."""
    T, H_q, D = q.shape
    num_pages, H_kv, ps, _ = k_cache.shape
    G = H_q // H_kv
    out = np.full((T, H_q, D), np.nan)
    mag, smax, cnt = np.zeros((T, H_q, D)), np.zeros((T, H_q)), np.zeros(T, dtype=np.int64)
    for b in range(len(kv_len)):
        L, n = int(kv_len[b]), int(cu[b + 1]) - int(cu[b])
        if n <= 0:
            continue
        k, ok = gather(k_cache, table[b], L, ps, num_pages)
        v, _ = gather(v_cache, table[b], L, ps, num_pages)
        for i in range(n):
            t = int(cu[b]) + i
            j = seen(L, n, i, window, sinks)
            j = j[ok[j]]
            cnt[t] = len(j)
            if len(j) == 0:
                out[t] = 0.0
                continue
            for g in range(H_kv):
                kk, vv, qq = k[j, g], v[j, g], q[t, g * G:(g + 1) * G]
                with np.errstate(all="ignore"):
                    s = scale * (qq @ kk.T)
                    e = np.exp(s - s.max(axis=1, keepdims=True))
                    p = e / e.sum(axis=1, keepdims=True)
                    out[t, g * G:(g + 1) * G] = p @ vv
                    mag[t, g * G:(g + 1) * G] = p @ np.abs(vv)
                    smax[t, g * G:(g + 1) * G] = scale * (np.abs(qq) @ np.abs(kk).T).max(axis=1)
    return out, mag, smax, cnt
