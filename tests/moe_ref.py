"""Plain 64-bit definitions of the operators around the expert products, for
the tests (numpy; nothing here calls the library)."""
import numpy as np


def route(x, topk, mask=None, normalize=False):
    """x [T, E] float64 (may hold -inf, NaN, +inf).  Returns a dict of the
    routing and p."""
    T, E = x.shape
    x = x.astype(np.float64).copy()
    if mask is not None:
        x[mask == 0] = -np.inf
    p = np.zeros((T, E))
    experts = np.full((T, topk), -1, np.int64)
    weights = np.zeros((T, topk))
    for t in range(T):
        row = x[t]
        bad = np.isnan(row).any() or (row == np.inf).any()
        if bad:
            p[t] = np.nan
        elif (row > -np.inf).any():
            e = np.exp(row - row.max())
            p[t] = e / e.sum()
        cand = [e for e in range(E) if row[e] > -np.inf]  # NaN compares false
        cand.sort(key=lambda e: (-row[e], e))
        for j, e in enumerate(cand[:topk]):
            experts[t, j] = e
            weights[t, j] = p[t, e]
        if normalize and cand:
            n = len(cand[:topk])
            weights[t, :n] /= weights[t, :n].sum()
    counts = np.bincount(experts[experts >= 0], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    slot_row = np.full((T, topk), -1, np.int64)
    row_index = np.full(T * topk, -1, np.int64)
    at = offsets[:-1].copy()
    for t in range(T):
        for j in range(topk):
            e = experts[t, j]
            if e >= 0:
                slot_row[t, j] = at[e]
                row_index[at[e]] = t
                at[e] += 1
    valid = T if mask is None else int((mask != 0).sum())
    prob_sum = p.sum(0)
    loss = E / (topk * valid * valid) * (counts * prob_sum).sum() if valid else 0.0
    return dict(p=p, experts=experts, weights=weights, counts=counts, group_offsets=offsets, slot_row=slot_row,
                row_index=row_index, valid=valid, prob_sum=prob_sum, loss=loss)


def route_objective(x, experts, counts, valid, dw, dl, normalize):
    """<dw, weights> + dl * loss with the choice and the counts held fixed, for
    difference quotients."""
    T, E = x.shape
    e = np.exp(x - x.max(1, keepdims=True))
    p = e / e.sum(1, keepdims=True)
    total = dl * E / (experts.shape[1] * valid * valid) * (counts * p.sum(0)).sum()
    for t in range(T):
        at = experts[t][experts[t] >= 0]
        w = p[t, at]
        if normalize:
            w = w / w.sum()
        total += (dw[t, : len(at)] * w).sum()
    return total


def route_backward(p, experts, counts, valid, dw, dl, normalize):
    """(d_x, size of the terms it is summed from)"""
    T, E = p.shape
    k = experts.shape[1]
    b = dl * E / (k * valid * valid) * counts if valid else np.zeros(E)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        slots = np.nonzero(experts[t] >= 0)[0]
        at, w = experts[t, slots], dw[t, slots]
        q = p[t, at].copy()
        if normalize and len(at):
            q = q / q.sum()
        qd, qa = (q * w).sum(), (q * np.abs(w)).sum()
        pb, pa = (p[t] * b).sum(), (p[t] * np.abs(b)).sum()
        if normalize:
            d[t] = p[t] * (b - pb)
            size[t] = p[t] * (np.abs(b) + pa)
            d[t, at] += q * (w - qd)
            size[t, at] += q * (np.abs(w) + qa)
        else:
            d[t] = p[t] * (b - pb - qd)
            size[t] = p[t] * (np.abs(b) + pa + qa)
            d[t, at] += q * w
            size[t, at] += q * np.abs(w)
    return d, size


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(h):
    c = h.shape[1] // 2
    g, u = h[:, :c], h[:, c:]
    return g * sigmoid(g) * u


def swiglu_backward(h, dy):
    c = h.shape[1] // 2
    g, u = h[:, :c], h[:, c:]
    s = sigmoid(g)
    return np.concatenate([dy * u * s * (1 + g * (1 - s)), dy * g * s], axis=1)


def wgrad(dy, x, offsets, row_index=None):
    """(dW [groups * N, K], sum of |products|, rows of each group)"""
    src = x if row_index is None else x[row_index]
    out, mag, n = [], [], []
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        out.append(dy[lo:hi].T @ src[lo:hi])
        mag.append(np.abs(dy[lo:hi]).T @ np.abs(src[lo:hi]))
        n.append(hi - lo)
    return np.concatenate(out), np.concatenate(mag), np.array(n)


def combine(y, slot_row, w):
    T, k = slot_row.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < len(y):
                out[t] += w[t, j] * y[r]
                mag[t] += np.abs(w[t, j] * y[r])
    return out, mag
