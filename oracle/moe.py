"""Plain NumPy expert routing and expert row layout, token by token, in 64 bits.

Routing: scores softmax(x) or 1 / (1 + exp(-x)), a logit of -inf switching its expert off; the choice goes
by score + bias (for softmax without bias and groups judged by one expert: by the logit) within the best
groups, ties to the lower index; weights are the chosen scores, renormalised or not, times a scale.
Layout: the (token, k) entries of each expert in order, at 128-aligned starts (contiguous) or a fixed pitch
(masked).
"""

import numpy as np


def scores(x, score):
    """Scores of one token's logits (experts,), 0 where the logit is -inf."""
    x = np.asarray(x, dtype=np.float64)
    free = x != -np.inf
    s = np.zeros_like(x)
    if not free.any():
        return s
    if score == "softmax":
        s[free] = np.exp(x[free] - x[free].max())
        return s / s.sum()
    s[free] = 1.0 / (1.0 + np.exp(-x[free]))
    return s


def choice_values(x, score, bias=None, num_groups=1, group_top=1):
    """What one token's experts are compared by; -inf: not available."""
    x = np.asarray(x, dtype=np.float64)
    if score == "softmax" and bias is None and not (num_groups > 1 and group_top > 1):
        return x.copy()
    v = scores(x, score) + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    v[x == -np.inf] = -np.inf
    return v


def kept_groups(values, num_groups, topk_groups, group_top):
    """Experts (bool mask) of the topk_groups best groups."""
    of_group = values.reshape(num_groups, -1)
    total = np.full(num_groups, -np.inf)
    for g in range(num_groups):
        best = np.sort(of_group[g][of_group[g] != -np.inf])[::-1][:group_top]
        if best.size:
            total[g] = best.sum()
    keep = np.argsort(-total, kind="stable")[:topk_groups]
    mask = np.zeros(num_groups, dtype=bool)
    mask[keep] = True
    return np.repeat(mask, of_group.shape[1])


def route(logits, top_k, bias=None, num_groups=1, topk_groups=1, group_top=1, score="softmax", renormalize=True,
          scale=1.0):
    """(ids int32 (T, top_k), weights float64 (T, top_k))."""
    logits = np.asarray(logits, dtype=np.float64)
    t = logits.shape[0]
    ids = np.full((t, top_k), -1, dtype=np.int32)
    weights = np.zeros((t, top_k))
    for i in range(t):
        v = choice_values(logits[i], score, bias, num_groups, group_top)
        if num_groups > 1:
            v[~kept_groups(v, num_groups, topk_groups, group_top)] = -np.inf
        order = np.argsort(-v, kind="stable")[:top_k]
        order = order[v[order] != -np.inf]
        ids[i, :order.size] = order
    return ids, weights_of(logits, ids, score, renormalize, scale)


def weights_of(logits, ids, score, renormalize, scale):
    """The weights of a given choice."""
    logits = np.asarray(logits, dtype=np.float64)
    w = np.zeros(ids.shape)
    for i in range(ids.shape[0]):
        there = ids[i] >= 0
        s = scores(logits[i], score)[ids[i][there]]
        if renormalize:
            # relative to the chosen alone, so that it has a value where every score underflows
            if score == "softmax" and s.size:
                xk = logits[i][ids[i][there]]
                s = np.exp(xk - xk.max())
            s = s / s.sum() if s.sum() > 0 else np.zeros_like(s)
        w[i][there] = scale * s
    return w


def route_grad(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """dL/dlogits (T, E) of L = sum(dweights * weights) with the choice held fixed."""
    logits = np.asarray(logits, dtype=np.float64)
    dweights = np.asarray(dweights, dtype=np.float64)
    dx = np.zeros_like(logits)
    for i in range(ids.shape[0]):
        there = ids[i] >= 0
        pick, g = ids[i][there], dweights[i][there]
        if not pick.size:
            continue
        s = scores(logits[i], score)
        ds = np.zeros_like(s)
        if renormalize:
            total = s[pick].sum()
            if total == 0:
                continue
            ds[pick] = scale * (g - (s[pick] / total * g).sum()) / total
        else:
            ds[pick] = scale * g
        dx[i] = s * (ds - (s * ds).sum()) if score == "softmax" else ds * s * (1.0 - s)
    return dx


def layout(ids, num_experts, rows_per_expert=0, align=128):
    """(rows (T, K), sources (rows,), m_indices or None, counts): rows of the contiguous layout end with
    the last expert's."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    rows = np.full(flat.size, -1, dtype=np.int32)
    counts = np.zeros(num_experts, dtype=np.int32)
    sources, m_indices = [], []
    for e in range(num_experts):
        who = np.flatnonzero(flat == e)
        counts[e] = who.size
        if rows_per_expert:
            who = who[:rows_per_expert]
            length = rows_per_expert
        else:
            length = -(-who.size // align) * align
        rows[who] = len(sources) + np.arange(who.size)
        sources += who.tolist() + [-1] * (length - who.size)
        m_indices += [e] * length
    return (rows.reshape(ids.shape), np.array(sources, dtype=np.int32),
            None if rows_per_expert else np.array(m_indices, dtype=np.int32), counts)


def dispatch(x, sources, top_k):
    """x (T, H) -> rows (zeros where no entry is)."""
    out = np.zeros((len(sources), x.shape[1]), dtype=x.dtype)
    used = sources >= 0
    out[used] = x[sources[used] // top_k]
    return out


def combine(out, rows, weights=None):
    """y (T, H) in float64."""
    t, k = rows.shape
    y = np.zeros((t, out.shape[1]))
    for i in range(t):
        for j in range(k):
            if rows[i, j] >= 0:
                y[i] += (1.0 if weights is None else float(weights[i, j])) * out[rows[i, j]].astype(np.float64)
    return y


def combine_grad(dy, out, rows, weights):
    """(dout (rows, H), dweights (T, K)) in float64."""
    dout = np.zeros(out.shape)
    dw = np.zeros(rows.shape)
    for i in range(rows.shape[0]):
        for j in range(rows.shape[1]):
            r = rows[i, j]
            if r >= 0:
                dout[r] = float(weights[i, j]) * dy[i].astype(np.float64)
                dw[i, j] = (dy[i].astype(np.float64) * out[r].astype(np.float64)).sum()
    return dout, dw
