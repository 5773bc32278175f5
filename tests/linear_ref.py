"""Plain forms in 64 bits of linear attention with a fixed decay, token probabilities and draft acceptance, for the tests."""
import numpy as np
import torch


def power(log_decay, e):
    """g^e per head; g^0 is 1 for g = 0 too."""
    ld = log_decay.double()
    return torch.ones_like(ld) if e == 0 else torch.exp(ld * e)


def steps(S, q, k, v, log_decay, scale):
    """Token by token from S [HV, DV, DK]: (o [n, HV, DV], the states after every token, and sums of absolute values: of o's terms
    and of the state's)."""
    G = v.shape[1] // k.shape[1]
    S, q, k, v = S.double(), q.double().repeat_interleave(G, 1), k.double().repeat_interleave(G, 1), v.double()
    A, g = S.abs(), power(log_decay, 1)[:, None, None]
    o, states, oa, sa = [], [], [], []
    for t in range(v.shape[0]):
        S = (torch.where(g == 0, torch.zeros_like(S), g * S)) + v[t][:, :, None] * k[t][:, None, :]
        A = (torch.where(g == 0, torch.zeros_like(A), g * A)) + v[t].abs()[:, :, None] * k[t].abs()[:, None, :]
        o.append(scale * (S @ q[t][:, :, None]).squeeze(-1))
        oa.append(abs(scale) * (A @ q[t].abs()[:, :, None]).squeeze(-1))
        states.append(S)
        sa.append(A)
    n = v.shape[0]
    shape = (n, v.shape[1], v.shape[2])
    empty = torch.zeros(shape, dtype=torch.float64)
    return (torch.stack(o) if n else empty, states, torch.stack(oa) if n else empty, sa)


def softmax(x, T):
    """Probabilities of one row of logits (float64 numpy), and the magnitude of the exponents."""
    out, mag = np.zeros_like(x), np.zeros_like(x)
    if np.isnan(x).any() or (x == np.inf).any() or not (0 <= T < np.inf) or not np.isfinite(x).any():
        return out, mag
    m = x.max()
    if T < 2.0 ** -126:
        out[int(np.argmax(x))] = 1
        return out, mag
    with np.errstate(over="ignore"):
        d = (x - m) / T
        e = np.exp(d)
    return e / e.sum(), np.where(np.isfinite(d), np.abs(d), 0) / np.log(2)


def accept(p, q, drafts, u):
    """One lane: p [T, V], q [T - 1, V] or None, drafts [T - 1], u [T] -> (accept_len, tokens)."""
    T, V = p.shape
    p = p.astype(np.float64)
    n = 0
    while n < T - 1:
        x = int(drafts[n])
        if not 0 <= x < V:
            break
        qx = 1.0 if q is None else float(q[n, x])
        if not float(u[n]) * qx < p[n, x]:
            break
        n += 1
    row = np.where(np.isfinite(p[n]), p[n], 0.0)
    r = row
    if n < T - 1 and 0 <= int(drafts[n]) < V:
        other = np.zeros(V) if q is None else q[n].astype(np.float64)
        if q is None:
            other[int(drafts[n])] = 1.0
        bad = ~np.isfinite(other) | ~np.isfinite(p[n])
        r = np.where(bad, 0.0, np.maximum(row - np.where(bad, 0, other), 0.0))
        if not r.sum() > 0:
            r = np.maximum(row, 0.0)
    r = np.maximum(r, 0.0)
    token = -1
    if r.sum() > 0:
        c = np.cumsum(r)
        hit = np.flatnonzero((c > float(u[T - 1]) * c[-1]) & (r > 0))
        token = int(hit[0]) if len(hit) else int(np.flatnonzero(r > 0)[-1])
    return n + 1, [int(drafts[i]) for i in range(n)] + [token] + [-1] * (T - 1 - n)
