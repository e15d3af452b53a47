"""Products whose matrix depends on the row: the row plan, the top-k router,
the expert products and the low-rank adapters, in plain loops and fp64."""
import numpy as np


def group_rows(ids, groups):
    """(offsets, order, pos): rows sorted by id, equal ids in row order; rows
    whose id is outside [0, groups) are left out (order padded with -1, pos -1)."""
    ids = np.asarray(ids).reshape(-1)
    order, offsets = [], [0]
    for g in range(groups):
        order += [i for i in range(len(ids)) if ids[i] == g]
        offsets.append(len(order))
    pos = np.full(len(ids), -1, np.int32)
    for at, i in enumerate(order):
        pos[i] = at
    order = np.array(order + [-1] * (len(ids) - len(order)), np.int32)
    return np.array(offsets, np.int32), order, pos


def moe_route(logits, top_k, renorm):
    """(ids, weights fp64): per token the top_k largest logits (ties: the
    lowest expert), softmax weights over the chosen or over all.  -inf and NaN
    are never chosen; +inf counts as the largest finite fp32."""
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    ids = np.full((l.shape[0], top_k), -1, np.int32)
    weights = np.zeros((l.shape[0], top_k))
    for t in range(l.shape[0]):
        left = [e for e in range(l.shape[1]) if l[t, e] > -np.inf]
        if not left:
            continue
        top = max(l[t, e] for e in left)
        total = sum(np.exp(l[t, e] - top) for e in left)
        chosen = sorted(left, key=lambda e: (-l[t, e], e))[:top_k]
        p = np.array([np.exp(l[t, e] - top) for e in chosen])
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = p / (p.sum() if renorm else total)
    return ids, weights


def y_experts(codes, s_w, x, offsets, order, per_row, s_x=None):
    """Product rows [rows][n] in the plan's order (rows behind the last group
    are NaN); order None: x is in the plan's order.  x fp64-able [x_rows][k]."""
    codes = np.asarray(codes, np.float64)
    x = np.asarray(x, np.float64)
    rows = len(order) if order is not None else x.shape[0]
    y = np.full((rows, codes.shape[1]), np.nan)
    for g in range(codes.shape[0]):
        lo, hi = offsets[g], offsets[g + 1]
        if lo == hi:
            continue
        src = np.arange(lo, hi) if order is None else np.asarray(order[lo:hi]) // per_row
        p = (x[src] @ codes[g].T) / np.asarray(s_w[g], np.float64)
        y[lo:hi] = p if s_x is None else p / np.asarray(s_x, np.float64)[src][:, None]
    return y


def y_swiglu(gate, up):
    """gate / (1 + exp(-gate)) * up (fp64; the limit -0 for gates far below 0)."""
    with np.errstate(over="ignore"):
        return gate / (1.0 + np.exp(-gate)) * up


def y_combine(y, pos, weights):
    """[tokens][n]: sum over the slots of weights * y[pos] (pos -1: nothing)."""
    pos = np.asarray(pos).reshape(np.asarray(weights).shape)
    out = np.zeros((pos.shape[0], y.shape[1]))
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if pos[t, j] >= 0:
                out[t] += float(weights[t, j]) * y[pos[t, j]]
    return out


def lora_delta(x, ids, a, b, scale):
    """scale[g] B[g] (A[g] x[t]) per row t with g = ids[t] (zero rows outside)."""
    x = np.asarray(x, np.float64)
    out = np.zeros((x.shape[0], b.shape[1]))
    for t in range(x.shape[0]):
        g = int(ids[t])
        if 0 <= g < a.shape[0]:
            out[t] = (1.0 if scale is None else float(scale[g])) * (np.asarray(b[g], np.float64) @
                                                                   (np.asarray(a[g], np.float64) @ x[t]))
    return out
