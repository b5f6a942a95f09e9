"""Plain numpy definitions, in 64 bits, of the draft-model calls: top-logit
lists, the distillation loss and its gradient, beam selection and reordering.
Test infrastructure only; it shares no code with the library.

Logits come as float arrays whose values are the inputs' own (a bfloat16
tensor widened).  An entry at or below -1e30, or a NaN, is masked.
"""
import numpy as np

MASKED = -1e30


def visible(x):
    with np.errstate(invalid="ignore"):
        return np.asarray(x, np.float64) > MASKED


def log_sum_exp(z, seen):
    """ln of the sum of e^z over the seen entries (-inf without any)."""
    if not seen.any():
        return -np.inf
    m = z[seen].max()
    return m + np.log(np.exp(z[seen] - m).sum())


def row_topk(x, k, T=1.0):
    """values, ids and log-normalisers of a [rows, V] array."""
    x = np.asarray(x)
    R, V = x.shape
    values = np.full((R, k), -np.inf)
    ids = np.full((R, k), -1, np.int32)
    lse = np.full(R, -np.inf)
    for r in range(R):
        seen = visible(x[r])
        at = np.flatnonzero(seen)
        order = at[np.argsort(-x[r][at].astype(np.float64), kind="stable")][:k]
        values[r, :len(order)] = x[r][order]
        ids[r, :len(order)] = order
        lse[r] = log_sum_exp(x[r].astype(np.float64) / T, seen)
    return values, ids, lse


def distill(student, ids, logits, lse, T=1.0, keep=None, grad_loss=None):
    """Per-row loss [R] and gradient [R, V] (with the upstream gradient)."""
    x = np.asarray(student, np.float64)
    R, V = x.shape
    loss = np.zeros(R)
    grad = np.zeros((R, V))
    g = np.ones(R) if grad_loss is None else np.asarray(grad_loss, np.float64)
    for r in range(R):
        if keep is not None and not keep[r]:
            continue
        listed = [(int(i), float(t)) for i, t in zip(ids[r], logits[r])
                  if 0 <= i < V and t > MASKED]
        seen = visible(x[r])
        if not listed or not seen.any():
            continue
        at = np.array([i for i, _ in listed])
        # relative to the largest logits, so that nothing is lost however large l/T
        t = np.array([v for _, v in listed])
        if lse is None:
            t = (t - t.max()) / T
            norm = log_sum_exp(t, np.ones(len(t), bool))
        else:
            t, norm = t / T, float(lse[r])
        p = np.exp(t - norm)
        z = (np.where(seen, x[r], 0.0) - x[r][seen].max()) / T
        log_total = log_sum_exp(z, seen)
        log_q = np.where(seen, z - log_total, -np.inf)
        q = np.exp(log_q)
        outside = seen.copy()
        outside[at] = False
        rest = 0.0
        log_rho = -np.inf
        if lse is not None and outside.any():
            rest = max(0.0, 1.0 - p.sum())
            log_rho = log_sum_exp(z, outside) - log_total
        some = p > 0
        with np.errstate(divide="ignore", invalid="ignore"):
            loss[r] = (p[some] * (t[some] - norm - log_q[at[some]])).sum()
            if rest > 0:
                loss[r] += rest * (np.log(rest) - log_rho)
        d = q * (p.sum() + rest)
        if rest > 0:
            d[outside] -= rest * np.exp(log_q[outside] - log_rho)
        np.subtract.at(d, at, p)
        grad[r] = d * g[r] / T
    return loss, grad


def beam_select(x, scores, n, T=1.0, ended=None, eos=-1):
    """scores, parents, tokens, ended [B, n] of [B, W, V] logits."""
    x = np.asarray(x, np.float64)
    B, W, V = x.shape
    out = np.full((B, n), -np.inf)
    parents = np.full((B, n), -1, np.int32)
    tokens = np.full((B, n), -1, np.int32)
    over = np.zeros((B, n), np.uint8)
    for b in range(B):
        cand = []
        for w in range(W):
            s = float(scores[b, w])
            if not s > -np.inf:
                continue
            if ended is not None and ended[b, w]:
                cand.append((-s, w, eos, 0))
                continue
            seen = visible(x[b, w])
            if not seen.any():
                continue
            z = (np.where(seen, x[b, w], 0.0) - x[b, w][seen].max()) / T
            norm = log_sum_exp(z, seen)
            at = np.flatnonzero(seen)
            order = at[np.argsort(-x[b, w][at], kind="stable")][:n]
            # a row's own candidates are ordered by their logits, then ids
            cand += [(-(s + (z[i] - norm)), w, int(i), c) for c, i in enumerate(order)]
        cand.sort(key=lambda c: (c[0], c[1], c[3]))
        for i, (key, w, tok, _) in enumerate(cand[:n]):
            out[b, i], parents[b, i], tokens[b, i] = -key, w, tok
            over[b, i] = int((ended is not None and ended[b, w] != 0) or tok == eos)
    return out, parents, tokens, over


def beam_reorder(parents, src, dst, lengths=None):
    """dst [B, n, segments, positions, ...] with the used positions of each
    beam's parent copied in; a parent outside the beams leaves its row."""
    src = np.array(src, copy=True)
    out = np.array(dst, copy=True)
    B, n = parents.shape
    for b in range(B):
        used = src.shape[3] if lengths is None else min(max(int(lengths[b]), 0), src.shape[3])
        for i in range(n):
            w = int(parents[b, i])
            if 0 <= w < src.shape[1]:
                out[b, i, :, :used] = src[b, w, :, :used]
    return out
