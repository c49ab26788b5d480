"""Oracle of the paged-cache operators: TEST INFRASTRUCTURE ONLY (tests and smoke may use it;
the CUDA library never does).  Plain numpy in fp64, one token and one key at a time where
that states the rule best.

Readings taken here: position t of sequence b is slot t % page_size of page
table[b][t // page_size]; a page number outside the cache holds nothing; node n of tree b sits at
position prefix_len[b] + n and is rotated by prefix_len[b] + position_ids[b][n]; a query (b, n)
with n < counts[b] sees the positions before prefix_len[b] and the drafts its mask names;
what it does not see never reaches its result.
"""
import numpy as np


def slot(table_row, n_pages, page_size, t):
    """(page, slot) of position t, or None where nothing holds it."""
    if t < 0 or t // page_size >= len(table_row):
        return None
    page = int(table_row[t // page_size])
    return (page, t % page_size) if 0 <= page < n_pages else None


def rotate(x, row, interleaved):
    """x [..., head_dim] (fp64) rotated by a cos_sin row [rot_dim]."""
    rot = len(row)
    h = rot // 2
    out = np.array(x, dtype=np.float64)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        out[..., a] = x[..., a] * row[i] - x[..., b] * row[h + i]
        out[..., b] = x[..., b] * row[i] + x[..., a] * row[h + i]
    return out


def append(q, k, v, k_cache, v_cache, table, prefix_len, cos_sin, position_ids=None, counts=None,
           interleaved=False):
    """Returns (rotated queries, key cache, value cache) in fp64."""
    B, N = k.shape[:2]
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    out = np.zeros(q.shape)
    n_pages, page_size = kc.shape[:2]
    for b in range(B):
        pre = max(int(prefix_len[b]), 0)
        for n in range(N):
            if counts is not None and n >= counts[b]:
                continue
            r = pre + (n if position_ids is None else int(position_ids[b][n]))
            if cos_sin.shape[1] and not 0 <= r < len(cos_sin):
                continue
            row = cos_sin[r] if cos_sin.shape[1] else cos_sin.reshape(-1)[:0]
            out[b, n] = rotate(q[b, n].astype(np.float64), row.astype(np.float64), interleaved)
            at = slot(table[b], n_pages, page_size, pre + n)
            if at is not None:
                kc[at] = rotate(k[b, n].astype(np.float64), row.astype(np.float64), interleaved)
                vc[at] = v[b, n]
    return out, kc, vc


def attention(q, k_cache, v_cache, table, prefix_len, scale, mask=None, counts=None,
              shared_len=0):
    """Returns out, lse, and for the tests' tolerances: sum_t p_t |v_t| and the largest
    scale * sum_i |q_i| |k_i| over the visible keys."""
    B, N, Hq, D = q.shape
    n_pages, page_size, Hkv = k_cache.shape[:3]
    G = Hq // Hkv
    out, mag = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse, size = np.full((B, N, Hq), -np.inf), np.zeros((B, N, Hq))
    for b in range(B):
        pre = max(int(prefix_len[b]), 0)
        cnt = N if counts is None else min(max(int(counts[b]), 0), N)
        if pre < shared_len:
            continue
        for n in range(cnt):
            seen = list(range(pre))
            seen += [pre + j for j in range(cnt) if (j <= n if mask is None else mask[b][n][j])]
            at = [slot(table[0 if t < shared_len else b], n_pages, page_size, t) for t in seen]
            at = [x for x in at if x is not None]
            if not at:
                continue
            pg, sl = np.array(at).T
            for h in range(Hq):
                K = k_cache[pg, sl, h // G].astype(np.float64)
                V = v_cache[pg, sl, h // G].astype(np.float64)
                x = q[b, n, h].astype(np.float64)
                with np.errstate(invalid="ignore"):
                    s = scale * (K @ x)
                    p = np.exp(s - s.max())
                    out[b, n, h] = (p[:, None] * V).sum(0) / p.sum()
                    mag[b, n, h] = (p[:, None] * np.abs(V)).sum(0) / p.sum()
                    lse[b, n, h] = s.max() + np.log(p.sum())
                    size[b, n, h] = abs(scale) * (np.abs(K) @ np.abs(x)).max()
    return out, lse, mag, size


def commit(cache, table, prefix_len, accepted_path, accept_len):
    """cache [planes, n_pages, page_size, heads, row]; returns the committed copy."""
    out = np.array(cache, copy=True)
    n_pages, page_size = out.shape[1:3]
    for b in range(len(prefix_len)):
        pre = max(int(prefix_len[b]), 0)
        for k in range(1, int(accept_len[b]) + 1):
            src = slot(table[b], n_pages, page_size, pre + int(accepted_path[b][k]))
            dst = slot(table[b], n_pages, page_size, pre + k)
            if src is not None and dst is not None:
                out[:, dst[0], dst[1]] = out[:, src[0], src[1]]
    return out
