"""Plain float64 oracle of the operators around the decode step (test infrastructure
only): the layer's inputs, the scan of packed prompts and the gated norm, token by token
in numpy. It shares no code with the CUDA path."""

from __future__ import annotations

import numpy as np


def silu(x):
    with np.errstate(over="ignore", invalid="ignore"):
        return x / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(x, 0.0)


def rows_served(cu, seqs, n_rows):
    """(sequence, begin, end, row) of the sequences that are served: padding, ids past the
    state and all but the first of equal ids are left out."""
    seen, out = set(), []
    for s in range(len(cu) - 1):
        row = s if seqs is None else int(seqs[s])
        if row < 0 or row >= n_rows or row in seen:
            continue
        seen.add(row)
        out.append((s, int(cu[s]), int(cu[s + 1]), row))
    return out


def prompt_inputs(x, raw, w, bias, dt_bias, A, conv, cu, seqs=None, resume=None):
    """Channels [T][D] convolved and gated (not split), dt, a [T][H], the new state, and the
    sum of the magnitudes of each convolution's terms (for error bounds). Tokens that no
    sequence owns are NaN."""
    K, D = w.shape[0] - 1, w.shape[1]
    y, mag = np.full((x.shape[0], D), np.nan), np.full((x.shape[0], D), np.nan)
    dt, a = np.full((x.shape[0], A.shape[0]), np.nan), np.full((x.shape[0], A.shape[0]), np.nan)
    conv = conv.copy()
    b = np.zeros(D) if bias is None else bias
    for s, t0, t1, row in rows_served(cu, seqs, conv.shape[0]):
        old = conv[row] if resume is not None and resume[s] else np.zeros((K, D))
        seen = np.concatenate([old, x[t0:t1]])
        for t in range(t0, t1):
            taps = w * seen[t - t0:t - t0 + K + 1]
            y[t] = silu(taps.sum(0) + b)
            mag[t] = np.abs(taps).sum(0) + np.abs(b)
        conv[row] = seen[len(seen) - K:]
        dt[t0:t1] = softplus(raw[t0:t1] + (0.0 if dt_bias is None else dt_bias))
        a[t0:t1] = np.exp(-dt[t0:t1] * A)
    return y, dt, a, conv, mag


def split(y, H, G, P, N):
    """Channels [T][D] as q, k [T][G][N] and v [T][H][P]."""
    v, k, q = np.split(y, [H * P, H * P + G * N], axis=1)
    return q.reshape(-1, G, N), k.reshape(-1, G, N), v.reshape(-1, H, P)


def prompt_scan(q, k, v, dt, a, S, cu, seqs=None, resume=None):
    """y [T][H][P] and the new states [rows][H][P][N], token by token. Tokens that no sequence
    owns are NaN."""
    H, G = v.shape[1], q.shape[1]
    y = np.full(v.shape, np.nan)
    S = S.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        for s, t0, t1, row in rows_served(cu, seqs, S.shape[0]):
            X = S[row].copy() if resume is not None and resume[s] else np.zeros_like(S[row])
            for t in range(t0, t1):
                kt, qt = np.repeat(k[t], H // G, axis=0), np.repeat(q[t], H // G, axis=0)
                X = a[t][:, None, None] * X + (dt[t][:, None] * v[t])[:, :, None] * kt[:, None, :]
                y[t] = np.einsum("hpn,hn->hp", X, qt)
            S[row] = X
    return y, S


def prompt_scan_magnitude(q, k, v, dt, a, S, cu, seqs=None, resume=None):
    """The scan of the operands' magnitudes: what a forward error bound multiplies."""
    return prompt_scan(np.abs(q), np.abs(k), np.abs(v), np.abs(dt), np.abs(a), np.abs(S), cu, seqs, resume)


def gated_norm(y, z, weight, v=None, D=None, groups=1, eps=1e-5):
    """out [T][H*P]."""
    T = y.shape[0]
    u = y if v is None else y + D[None, :, None] * v
    u = (u.reshape(T, -1) * silu(z)).reshape(T, groups, -1)
    u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return u.reshape(T, -1) * weight
