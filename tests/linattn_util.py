"""Plain references for linear attention with a decay and for drafted trees
(not collected by pytest): the definitions of ikbo.h, row by row in 64 bits."""
from __future__ import annotations

import numpy as np

D = 128


def forward(Q, K, V, decay, offsets, S0, scale):
    """O [rows, H, D] (zero for rows of no user) and the last states; Q may be None, S0 too."""
    H, U = K.shape[1], len(offsets) - 1
    O = np.zeros(K.shape)
    S = np.zeros((U, H, D, D)) if S0 is None else np.array(S0, dtype=np.float64)
    lam = np.asarray(decay, dtype=np.float64)[:, None, None]
    for u in range(U):
        for r in range(offsets[u], offsets[u + 1]):
            S[u] = lam * S[u] + K[r][:, :, None] * V[r][:, None, :]
            if Q is not None:
                O[r] = scale * np.einsum("hd,hde->he", Q[r], S[u])
    return O, S


def backward(Q, K, V, dO, decay, offsets, S0, dS, scale):
    """dQ, dK, dV and the gradient of the first states."""
    H, U = K.shape[1], len(offsets) - 1
    dQ, dK, dV = (np.zeros(K.shape) for _ in range(3))
    R = np.zeros((U, H, D, D)) if dS is None else np.array(dS, dtype=np.float64)
    lam = np.asarray(decay, dtype=np.float64)[:, None, None]
    S = np.zeros((U, H, D, D)) if S0 is None else np.array(S0, dtype=np.float64)
    for u in range(U):
        for r in range(offsets[u], offsets[u + 1]):
            S[u] = lam * S[u] + K[r][:, :, None] * V[r][:, None, :]
            dQ[r] = scale * np.einsum("he,hde->hd", dO[r], S[u])
        for r in range(offsets[u + 1] - 1, offsets[u] - 1, -1):
            R[u] = R[u] + scale * Q[r][:, :, None] * dO[r][:, None, :]
            dK[r] = np.einsum("he,hde->hd", V[r], R[u])
            dV[r] = np.einsum("hd,hde->he", K[r], R[u])
            R[u] = lam * R[u]
    return dQ, dK, dV, R


def weights(K, V, decay, offsets, S0):
    """The sums of the magnitudes that make up a state: the same scan of absolute values."""
    return forward(None, np.abs(K), np.abs(V), decay, offsets, None if S0 is None else np.abs(S0), 1.0)[1]


def sees(parents):
    """[Lq, Lq] truth of one draft: row i reads row j; rows that are not there read nothing."""
    L = len(parents)
    m = np.zeros((L, L), dtype=bool)
    for l, up in enumerate(parents):
        if up < -1 or up >= l or (up >= 0 and not m[up, up]):
            continue
        if up >= 0:
            m[l] = m[up]
        m[l, l] = True
    return m


def tree(Q, kv, K_new, V_new, parents, map_, H_kv, scale):
    """O, lse and the bound of O's error, row by row.

    The bound counts the roundings: each p to bf16 (2^-8 of the mass sum p |v|, of
    the history's rows and of the draft's), the history's O to bf16 (2^-8 of its
    part) and the output (2^-8); the scores' fp32 sums (2^-16 of the largest
    sum |q k|) and the exponentials' arguments (2^-20), each twice; and the history's
    log-sum-exp as an fp32 number (2^-22 of its magnitude, in the exponent)."""
    n, H, Lq, d = Q.shape
    O, lse, bound = np.zeros(Q.shape), np.full((n, H, Lq), -np.inf), np.zeros(Q.shape)
    for i in range(n):
        u = int(map_[i])
        if not 0 <= u < len(kv):
            continue
        m = sees(parents[i])
        for h in range(H):
            g = h // (H // H_kv)
            Kh, Vh = (x[:, g].astype(np.float64) for x in kv[u])
            for l in range(Lq):
                if not m[l, l]:
                    continue
                k = np.concatenate([Kh, K_new[i, m[l], g]]).astype(np.float64)
                v = np.concatenate([Vh, V_new[i, m[l], g]]).astype(np.float64)
                q = Q[i, h, l].astype(np.float64)
                s = scale * (k @ q)
                top = s.max()
                p = np.exp(s - top)
                O[i, h, l] = p @ v / p.sum()
                lse[i, h, l] = top + np.log(p.sum())
                mass = p @ np.abs(v) / p.sum()
                e = 2.0 ** -16 * scale * (np.abs(k) @ np.abs(q)).max() + 2.0 ** -20 + 2.0 ** -22 * (1 + np.abs(lse[i, h, l]))
                bound[i, h, l] = 2.0 ** -8 * mass * 2 + 2.0 ** -8 * np.abs(O[i, h, l]) + 2 * e * mass + 1e-30
    return O, lse, bound
