"""Float64 oracle of linear attention with a scalar decay for each head, token by token:

    S <- exp(log_g) S + k v^T,   o = S^T q

Plain NumPy, one (sequence, head) at a time, sharing no code with the library.
"""

import numpy as np


def linear_attention(q, k, v, log_g, h0=None, cu_seqlens=None):
    """q, k: [B, T, Hk, dk]; v: [B, T, H, dv]; log_g: [B, T, H] or [H]; h0: [N, H, dk, dv] or None.
    Returns (o [B, T, H, dv], hT [N, H, dk, dv]) in float64."""
    q, k, v, log_g = (np.asarray(x, dtype=np.float64) for x in (q, k, v, log_g))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    if cu_seqlens is None:
        spans = [(b, 0, T) for b in range(B)]
    else:
        cu = [int(c) for c in np.asarray(cu_seqlens)]
        if cu[0] != 0 or cu[-1] != T or any(a > b for a, b in zip(cu, cu[1:])):
            raise ValueError("malformed cu_seqlens")
        spans = [(0, a, b) for a, b in zip(cu, cu[1:])]
    o = np.zeros((B, T, H, dv))
    hT = np.zeros((len(spans), H, dk, dv))
    for n, (b, t0, t1) in enumerate(spans):
        for h in range(H):
            hk = h // (H // Hk)
            S = np.zeros((dk, dv)) if h0 is None else np.array(h0[n, h], dtype=np.float64)
            for t in range(t0, t1):
                lg = log_g[h] if log_g.ndim == 1 else log_g[b, t, h]
                S = np.exp(lg) * S + np.outer(k[b, t, hk], v[b, t, h])
                o[b, t, h] = S.T @ q[b, t, hk]
            hT[n, h] = S
    return o, hT
