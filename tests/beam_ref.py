"""Plain implementations of the beam search operators in 64 bits (numpy)."""

import numpy as np


def select(x, scores, n, finished=None, end_token=0, weights=None):
    """x [N * K, V] float64 (the logits widened exactly). Returns (scores
    float64, parents, tokens), each [N, n]."""
    N, K = scores.shape
    c = scores.astype(np.float64)
    w = np.ones((N, K)) if weights is None else weights.astype(np.float64)
    out_s = np.full((N, n), -np.inf)
    out_p = np.full((N, n), -1, np.int32)
    out_t = np.full((N, n), -1, np.int32)
    for i in range(N):
        rank, beam, logit, token, score = [], [], [], [], []
        for b in range(K):
            if not (np.isfinite(c[i, b]) and np.isfinite(w[i, b]) and w[i, b] > 0):
                continue
            if finished is not None and finished[i, b]:
                r, tok, val, s = np.array([c[i, b] * w[i, b]]), np.array([end_token]), np.zeros(1), np.array([c[i, b]])
            else:
                row = x[i * K + b]
                if row.size == 0 or not np.isfinite(row.max()):  # NaN, +inf or nothing but -inf
                    continue
                top = row.max()
                rest = np.log(np.exp(row - top).sum())  # apart from top, which may be as large as the type goes
                tok = np.nonzero(row > -np.inf)[0]
                if tok.size > n:
                    least = np.partition(row[tok], -n)[-n]
                    tok = tok[row[tok] >= least]
                val = row[tok] + 0.0
                pick = np.lexsort((tok, -val))[:n]
                tok, val = tok[pick], val[pick]
                s = c[i, b] + ((val - top) - rest)
                r = s * w[i, b]
            rank.append(r)
            beam.append(np.full(r.size, b))
            logit.append(val)
            token.append(tok)
            score.append(s)
        if not rank:
            continue
        rank, beam, logit, token, score = (np.concatenate(v) for v in (rank, beam, logit, token, score))
        pick = np.lexsort((token, -logit, beam, -rank))[:n]
        m = pick.size
        out_s[i, :m], out_p[i, :m], out_t[i, :m] = score[pick], beam[pick], token[pick]
    return out_s, out_p, out_t


def reorder(state, parents, batch_dim, seq_dim=None, lengths=None):
    """A reordered copy of `state` (numpy)."""
    N, K = parents.shape
    out = state.copy()
    src, dst = np.moveaxis(state, batch_dim, 0), np.moveaxis(out, batch_dim, 0)
    axis = None
    if lengths is not None:
        d, s = batch_dim % state.ndim, seq_dim % state.ndim
        axis = s + 1 if s < d else s  # where the positions are once the rows are in front
        axis -= 1  # of one row
    for i in range(N):
        for b in range(K):
            p = parents[i, b]
            if not 0 <= p < K:
                continue
            if lengths is None:
                dst[i * K + b] = src[i * K + p]
            else:
                cut = (slice(None),) * axis + (slice(0, max(0, int(lengths[i]))),)
                dst[i * K + b][cut] = src[i * K + p][cut]
    return out


def backtrace(tokens, parents, beams=None, lengths=None, pad=-1):
    T, N, K = tokens.shape
    M = beams.shape[1] if beams is not None else (lengths.shape[1] if lengths is not None else K)
    out = np.full((N, M, T), pad, np.int32)
    for i in range(N):
        for m in range(M):
            b = m if beams is None else int(beams[i, m])
            e = T if lengths is None else min(max(int(lengths[i, m]), 0), T)
            for t in range(e - 1, -1, -1):
                if not 0 <= b < K:
                    break
                out[i, m, t] = tokens[t, i, b]
                b = int(parents[t, i, b])
    return out
