"""Plain fp64 definitions of the operators around the paged cache: rotary
positions, attention of drafted trees, accumulated attention weights, eviction
and row moves.  Test infrastructure only."""
import numpy as np
import torch


def to_np(x):
    return x.detach().to("cpu", torch.float64).numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)


def rotate(x, positions, inv_freq, interleaved=False, attn_scale=1.0, inverse=False):
    """x (rows, heads, d) -> fp64."""
    x, f = to_np(x), to_np(inv_freq)
    h = f.size
    a = to_np(positions)[:, None] * f[None] * (-1.0 if inverse else 1.0)
    c, s = attn_scale * np.cos(a)[:, None], attn_scale * np.sin(a)[:, None]
    first = np.arange(h) * 2 if interleaved else np.arange(h)
    second = first + (1 if interleaved else h)
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def slot(table_row, page_size, t):
    t = np.asarray(t)
    return np.asarray(table_row)[t // page_size].astype(np.int64) * page_size + t % page_size


def tokens(cache, table_row, n):
    """The first n tokens of a request: (n, heads, d) fp64."""
    rows = cache.reshape(-1, *cache.shape[2:])
    return to_np(rows[torch.from_numpy(slot(table_row.cpu().numpy(), cache.shape[1], np.arange(n)))])


def attend(q, k, v, seen, sink, scale):
    """One request: q (n, hq, d), k / v (t, hkv, d), seen (n, t).  Returns O (n, hq, d),
    LSE (hq, n), P (hq, n, t) and the same O with |v| (for error bounds)."""
    q, k, v = to_np(q), to_np(k), to_np(v)
    n, hq, d = q.shape
    group = hq // k.shape[1]
    O, A = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    LSE, P = np.zeros((hq, n)), np.zeros((hq, n, k.shape[0]))
    for h in range(hq):
        s = (q[:, h] @ k[:, h // group].T) * scale
        s = np.where(seen, s, -np.inf)
        sg = -np.inf if sink is None else float(sink[h])
        top = np.maximum(s.max(1) if s.shape[1] else np.full(n, -np.inf), sg)
        for i in range(n):
            if top[i] == -np.inf:
                LSE[h, i] = -np.inf
                continue
            if top[i] == np.inf:
                LSE[h, i] = np.inf
                continue
            e = np.exp(s[i] - top[i])
            z = e.sum() + np.exp(sg - top[i])
            P[h, i] = e / z
            LSE[h, i] = top[i] + np.log(z)
        O[:, h], A[:, h] = P[h] @ v[:, h // group], P[h] @ np.abs(v[:, h // group])
    return O, LSE, P, A


def in_window(t, pos, first, last):
    seen = t <= pos
    return seen if last <= 0 else seen & ((t < first) | (t >= pos + 1 - last))


def tree_seen(parents, prefix, first=0, last=0):
    """(n, prefix + n) truth values: which cached tokens each node sees."""
    n = len(parents)
    anc, depth = np.zeros((n, n), bool), np.zeros(n, int)
    for i, p in enumerate(parents):
        if p >= 0:
            anc[i] = anc[p]
            depth[i] = depth[p] + 1
        anc[i, i] = True
    pos = prefix + depth
    key = np.concatenate([np.arange(prefix), pos])
    seen = np.concatenate([np.ones((n, prefix), bool), anc], 1)
    return seen & in_window(key[None], pos[:, None], first, last)


def evict(weights, length, budget, first, last):
    """Kept tokens of one weight row, increasing."""
    w = np.asarray(weights, np.float64)[:length]
    if length <= budget:
        return np.arange(length)
    keep = set(range(first)) | set(range(length - last, length))
    middle = [t for t in range(first, length - last)]
    # a NaN below every number; equal weights: the earlier token
    middle.sort(key=lambda t: (np.isnan(w[t]), 0.0 if np.isnan(w[t]) else -w[t], t))
    keep |= set(middle[:budget - first - last])
    return np.array(sorted(keep))
