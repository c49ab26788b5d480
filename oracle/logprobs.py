"""Oracle of the log probabilities of given tokens, the entropy and the most likely tokens of rows of
logits: TEST INFRASTRUCTURE ONLY (tests and smoke may use it; the CUDA library never does).

Readings taken here: softmax of z / T over the whole row, natural logarithms; a token outside the
vocabulary has log probability -inf; the k largest logits with ties to the lower index; a row number
outside the rows gives -inf, entropy 0, tokens -1 (status 4); a row holding NaN or +inf, or all
-inf, gives NaN, tokens -1 (status 1).
"""
import numpy as np


def _as_f64(row):
    row = np.asarray(row)
    if row.dtype == np.uint16:  # raw bf16 bits
        return (row.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return row.astype(np.float64)


def token_logprobs(logits, tokens=None, k=0, temperature=1.0, rows=None):
    """logits [n, V] (float32, or uint16 raw bf16 bits), tokens [R, G], rows [R].  Returns
    logprobs [R, G], entropy [R], top_tokens [R, k], top_logprobs [R, k], status [R]."""
    logits = np.atleast_2d(np.asarray(logits))
    n, V = logits.shape
    rows = np.arange(n) if rows is None else np.asarray(rows)
    R = len(rows)
    tokens = np.zeros((R, 0), dtype=np.int64) if tokens is None else np.asarray(tokens).reshape(R, -1)
    lp = np.full(tokens.shape, -np.inf)
    ent = np.zeros(R)
    top = np.full((R, k), -1, dtype=np.int64)
    top_lp = np.full((R, k), -np.inf)
    status = np.zeros(R, dtype=np.int32)
    for r in range(R):
        if not 0 <= rows[r] < n:
            status[r] = 4
            continue
        z = _as_f64(logits[rows[r]])
        m = z.max()
        if np.isnan(z).any() or np.isinf(m):
            status[r] = 1
            lp[r], ent[r], top_lp[r] = np.nan, np.nan, np.nan
            continue
        x = (z - m) / temperature
        w = np.exp(x)
        # the maximum's own weight apart: ln(1 + the rest) where one token holds nearly all
        rest = w.sum() - 1.0 if w.sum() > 2.0 else np.delete(w, int(np.argmax(z))).sum()
        logs = np.log1p(rest)
        with np.errstate(invalid="ignore"):
            wx = np.where(w > 0, w * x, 0.0)
        ent[r] = logs - wx.sum() / (1.0 + rest)
        for g, t in enumerate(tokens[r]):
            if 0 <= t < V:
                lp[r, g] = x[t] - logs
        order = np.lexsort((np.arange(V), -z))[:k]
        top[r] = order
        top_lp[r] = x[order] - logs
    return {"logprobs": lp, "entropy": ent, "top_tokens": top, "top_logprobs": top_lp, "status": status}
