"""fp64 oracle of linear attention with a per-head decay over packed sequences,
of its gradients, and of the 8-bit form of its states.

For every sequence and head, with a = exp(log_decay):
    S_t = a S_{t-1} + k_t v_t^T,   o_t = scale * q_t^T S_t.
``forward`` and ``backward`` evaluate the sums over pairs directly;
``recurrent`` walks the recurrence and pins them.
"""
import numpy as np


def _ranges(cu):
    return list(zip(cu[:-1], cu[1:]))


def _powers(g, n):
    """a^(t-s) for s <= t < n, zero above the diagonal (a^0 = 1 for a = 0 too)."""
    away = np.arange(n)[:, None] - np.arange(n)[None, :]
    return np.where(away > 0, np.exp(g * np.maximum(away, 1)), np.where(away == 0, 1.0, 0.0))


def _reach(g, n):
    """a^1 .. a^n."""
    return np.exp(g * np.arange(1, n + 1))


def _share(g, n):
    """a^(n-1) .. a^0."""
    return _powers(g, n)[-1] if n else np.zeros(0)


def forward(q, k, v, log_decay, cu, scale, S0=None):
    """q, k [T,H,d], v [T,H,dv], S0 [N,H,d,dv] -> o [T,H,dv] (zero outside the sequences) and the final states."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, H, d = q.shape
    dv, N = v.shape[2], len(cu) - 1
    o = np.zeros((T, H, dv))
    S = np.zeros((N, H, d, dv)) if S0 is None else np.array(S0, np.float64)
    for n, (a, b) in enumerate(_ranges(cu)):
        for h in range(H):
            if b <= a:
                continue
            g, L = float(log_decay[h]), b - a
            x, y, z = q[a:b, h], k[a:b, h], v[a:b, h]
            o[a:b, h] = scale * ((x @ y.T * _powers(g, L)) @ z + _reach(g, L)[:, None] * (x @ S[n, h]))
            S[n, h] = np.exp(g * L) * S[n, h] + (y * _share(g, L)[:, None]).T @ z
    return o, S


def recurrent(q, k, v, log_decay, cu, scale, S0=None):
    """The same by the recurrence, token by token."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, H, d = q.shape
    dv, N = v.shape[2], len(cu) - 1
    o = np.zeros((T, H, dv))
    S = np.zeros((N, H, d, dv)) if S0 is None else np.array(S0, np.float64)
    a = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    for n, (t0, t1) in enumerate(_ranges(cu)):
        for t in range(t0, t1):
            S[n] = a * S[n] + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hd,hde->he", q[t], S[n])
    return o, S


def magnitude(q, k, v, log_decay, cu, scale, S0=None):
    """scale * sum of the magnitudes of the terms of o, and of S: what roundings of the factors are relative to."""
    return forward(np.abs(q), np.abs(k), np.abs(v), log_decay, cu, abs(scale), None if S0 is None else np.abs(S0))


def backward(q, k, v, dO, log_decay, cu, scale, S0=None, dS=None):
    """dq, dk, dv (zero outside the sequences) and dS0."""
    q, k, v, dO = (np.asarray(x, np.float64) for x in (q, k, v, dO))
    H, d = q.shape[1:]
    dvw, N = v.shape[2], len(cu) - 1
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    S0 = np.zeros((N, H, d, dvw)) if S0 is None else np.asarray(S0, np.float64)
    dS = np.zeros((N, H, d, dvw)) if dS is None else np.asarray(dS, np.float64)
    dS0 = dS.copy()
    for n, (a, b) in enumerate(_ranges(cu)):
        if b <= a:
            continue
        for h in range(H):
            g, L = float(log_decay[h]), b - a
            x, y, z, w = q[a:b, h], k[a:b, h], v[a:b, h], scale * dO[a:b, h]
            P, reach, share = _powers(g, L), _reach(g, L)[:, None], _share(g, L)[:, None]
            pair = (w @ z.T) * P
            dq[a:b, h] = pair @ y + reach * (w @ S0[n, h].T)
            dk[a:b, h] = pair.T @ x + share * (z @ dS[n, h].T)
            dv[a:b, h] = ((x @ y.T) * P).T @ w + share * (y @ dS[n, h])
            dS0[n, h] = np.exp(g * L) * dS[n, h] + (reach * x).T @ w
    return dq, dk, dv, dS0


def store_q8(S):
    """Integers and scales of the rows of S (last dimension) in the 8-bit form."""
    S = np.asarray(S, np.float32)
    with np.errstate(all="ignore"):
        m = np.abs(S).max(-1)
        scale = (m.astype(np.float64) / 127).astype(np.float32)
        scale = np.where(scale < np.float32(2.0 ** -126), np.float32(0), scale)
        bad = ~np.isfinite(S).all(-1)
        scale = np.where(bad, np.float32(np.nan), scale)
        live = np.isfinite(scale) & (scale > 0)
        c = np.where(live[..., None], np.rint(S.astype(np.float64) / scale.astype(np.float64)[..., None]), 0)
    return c.astype(np.int8), scale


def load_q8(c, scale):
    """fp32 values of the 8-bit form."""
    with np.errstate(all="ignore"):
        return (c.astype(np.float64) * scale.astype(np.float64)[..., None]).astype(np.float32)
