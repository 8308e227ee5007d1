"""fp64 numpy reference of the rotary positions and of linear attention with a decay for each
head, token by token from the definitions (no chunks, no segments)."""
import numpy as np


def rotary(x, positions, frequencies, interleaved=False, first=0, scale=1.0, inverse=False):
    """x: [B, H, N, D]; positions [N] or [B, N]; frequencies [n] radians per position."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(frequencies, dtype=np.float64)
    n = f.shape[0]
    pos = np.broadcast_to(np.asarray(positions, dtype=np.float64), (x.shape[0], x.shape[2]))
    y = x.copy()
    for c in range(n):
        a, b = (first + 2 * c, first + 2 * c + 1) if interleaved else (first + c, first + n + c)
        t = (-pos if inverse else pos)[:, None, :] * f[c]
        y[..., a] = scale * (x[..., a] * np.cos(t) - x[..., b] * np.sin(t))
        y[..., b] = scale * (x[..., b] * np.cos(t) + x[..., a] * np.sin(t))
    return y


def _lengths(lengths, B, N):
    return [N] * B if lengths is None else [int(x) for x in lengths]


def linear_forward(q, k, v, log_decay, scale, initial=None, lengths=None):
    """(o, final state, states before each token [B, H, N, D, D])."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, H, N, D = q.shape
    with np.errstate(under="ignore"):
        lam = np.exp(np.asarray(log_decay, dtype=np.float64))
    o = np.zeros((B, H, N, D))
    S = np.zeros((B, H, D, D)) if initial is None else np.asarray(initial, dtype=np.float64).copy()
    before = np.zeros((B, H, N, D, D))
    for b, n in enumerate(_lengths(lengths, B, N)):
        for t in range(n):
            before[b, :, t] = S[b]
            S[b] = lam[:, None, None] * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hd,hde->he", q[b, :, t], S[b])
    return o, S, before


def linear_backward(q, k, v, do, log_decay, scale, initial=None, lengths=None, d_final=None):
    """(dq, dk, dv, d_initial): the reverse recurrence of G = dL/dS."""
    q, k, v, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, do))
    B, H, N, D = q.shape
    with np.errstate(under="ignore"):
        lam = np.exp(np.asarray(log_decay, dtype=np.float64))[:, None, None]
    _, _, before = linear_forward(q, k, v, log_decay, scale, initial, lengths)
    dq, dk, dv = (np.zeros((B, H, N, D)) for _ in range(3))
    G = np.zeros((B, H, D, D)) if d_final is None else np.asarray(d_final, dtype=np.float64).copy()
    for b, n in enumerate(_lengths(lengths, B, N)):
        for t in reversed(range(n)):
            S = lam * before[b, :, t] + k[b, :, t, :, None] * v[b, :, t, None, :]
            G[b] += scale * q[b, :, t, :, None] * do[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("hde,he->hd", S, do[b, :, t])
            dk[b, :, t] = np.einsum("hde,he->hd", G[b], v[b, :, t])
            dv[b, :, t] = np.einsum("hde,hd->he", G[b], k[b, :, t])
            G[b] = lam * G[b]
    return dq, dk, dv, G


def linear_step(q, k, v, log_decay, scale, pool, slots, out_slots):
    """(o, new pool) of one token a row; rows with a negative slot take no part."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    old = np.asarray(pool, dtype=np.float64)
    new, o = old.copy(), np.zeros(q.shape)
    lam = np.exp(np.asarray(log_decay, dtype=np.float64))[:, None, None]
    for b, (i, j) in enumerate(zip(slots, out_slots)):
        if i < 0 or j < 0:
            continue
        S = lam * old[i] + k[b, :, :, None] * v[b, :, None, :]
        new[j] = S
        o[b] = scale * np.einsum("hd,hde->he", q[b], S)
    return o, new
