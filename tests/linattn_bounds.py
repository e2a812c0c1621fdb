"""Bounds of every element of what linear attention computes, beside linattn_util (not collected by pytest).

An output in bf16 is a sum of terms (q.k decayed) v and q S.  On its way a term is rounded to bf16 once, its
product q.k with the decay or the state's element, by at most 2^-8 of its magnitude; the output is rounded
once, by 2^-8 of itself.  What else there is to it is small beside that: the state's own 2^-14 of its magnitudes
(test_gpu_linattn.py derives it) and fp32 sums of at most 256 terms, 2^-16.  With `mass` the sum of the terms'
magnitudes (the definition on absolute values), an element is off by at most
    2^-8 |o| + (2^-8 + 2^-8 2^-8 + 2^-14 + 2^-16) mass  <  2^-8 |o| + (2^-8 + 2^-12) mass,
where the third part of the middle bracket is the output's rounding of the first error."""
import numpy as np
import torch

import linattn_util as R


def host(t):
    return t.double().cpu().numpy()


def absolute(d):
    """The same data, of magnitudes."""
    a = lambda x: None if x is None else np.abs(x)  # noqa: E731
    return [a(x) for x in (d.Q, d.K, d.V, d.dO)], a(d.S), a(d.dS)


def forward(d, scale):
    """O, the last states, and the masses of both."""
    (Q, K, V, _), S, _ = absolute(d)
    return (*R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, scale), *R.forward(Q, K, V, d.decay, d.off, S, scale))


def backward(d, scale):
    """(dQ, dK, dV, d_state_in) and their masses."""
    rows, S, dS = absolute(d)
    return (R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, d.S, d.dS, scale),
            R.backward(*rows, d.decay, d.off, S, dS, scale))


def near(got, want, mass, what=""):
    """Every element of a bf16 tensor."""
    got = host(got)
    over = np.abs(got - want) - 2.0 ** -8 * np.abs(want) - (2.0 ** -8 + 2.0 ** -12) * mass - 1e-37
    assert np.all(over <= 0), (what, np.unravel_index(np.nanargmax(over), over.shape), float(np.nanmax(over)), bool(np.isnan(over).any()))


def near_state(got, want, mass, what=""):
    """Every element of a state: 2^-14 of its magnitudes."""
    over = np.abs(host(got) - want) - 2.0 ** -14 * mass - 1e-37
    assert np.all(over <= 0), (what, np.unravel_index(np.nanargmax(over), over.shape), float(np.nanmax(over)))


# ------------------------------------------------- the definition in chunks, for long histories, in torch's 64 bits
CHUNK = 128


def scan(x, y, z, lam, S, early, seen):
    """One user's rows [n, H, D] (x may be None), in order: out_t = x_t S_t with S_t = lam S_{t-1} + y_t z_t^T; early: S is
    before its first row's decay already.  Returns out, the end, and the largest element of a state at a chunk's border."""
    n, H, D = y.shape
    out = torch.zeros_like(y)
    lam = lam.double()[:, None, None]
    for c in range(0, n, CHUNK):
        k, v = y[c:c + CHUNK].transpose(0, 1), z[c:c + CHUNK].transpose(0, 1)
        m = k.shape[1]
        e = early if c == 0 else 0
        i = torch.arange(m, dtype=torch.float64, device=y.device)
        seen = max(seen, float(S.abs().max()))
        if x is not None:
            q = x[c:c + CHUNK].transpose(0, 1)
            gap = i[:, None] - i[None, :]
            w = torch.where(gap >= 0, lam ** gap.clamp(min=0), 0.0)
            out[c:c + CHUNK] = ((q @ k.transpose(1, 2) * w) @ v + lam ** (i + 1 - e)[:, None] * (q @ S)).transpose(0, 1)
        S = lam ** (m - e) * S + (k * lam ** (m - 1 - i)[:, None]).transpose(1, 2) @ v
    return out, S, max(seen, float(S.abs().max()))


def long_forward(Q, K, V, decay, off, S0, scale):
    """O, the last states, the largest element of one."""
    Q, K, V = (None if t is None else t.double() for t in (Q, K, V))
    U, H, D = len(off) - 1, K.shape[1], K.shape[2]
    O, S = torch.zeros_like(K), torch.zeros((U, H, D, D), dtype=torch.float64, device=K.device) if S0 is None else S0.double().clone()
    seen = 0.0
    for u in range(U):
        r = slice(int(off[u]), int(off[u + 1]))
        O[r], S[u], seen = scan(None if Q is None else Q[r], K[r], V[r], decay, S[u], 0, seen)
    return O * scale, S, seen


def long_backward(Q, K, V, dO, decay, off, S0, dS, scale):
    """dQ, dK, dV, the gradient of the first states, the largest element of a state."""
    Q, K, V, dO = (t.double() for t in (Q, K, V, dO))
    U, H, D = len(off) - 1, K.shape[1], K.shape[2]
    zero = torch.zeros((U, H, D, D), dtype=torch.float64, device=K.device)
    S0, R = zero if S0 is None else S0.double(), zero.clone() if dS is None else dS.double().clone()
    dQ, dK, dV, seen = torch.zeros_like(K), torch.zeros_like(K), torch.zeros_like(K), 0.0
    for u in range(U):
        r = slice(int(off[u]), int(off[u + 1]))
        if off[u] == off[u + 1]:
            continue
        dQ[r], _, seen = scan(dO[r], V[r], K[r], decay, S0[u].transpose(1, 2), 0, seen)
        q, k, v, do = (t[r].flip(0) for t in (Q * scale, K, V, dO))
        a, _, seen = scan(v, do, q, decay, R[u].transpose(1, 2), 1, seen)
        b, end, seen = scan(k, q, do, decay, R[u], 1, seen)
        dK[r], dV[r], R[u] = a.flip(0), b.flip(0), end * decay.double()[:, None, None]
    return dQ * scale, dK, dV, R, seen


def near_blocks(got, want, off, what=""):
    """The 2-norm of each user's 128 rows at a time and each head: independent roundings come to less than 2^-8 of it."""
    err, want = got.double() - want, want.double()
    for u in range(len(off) - 1):
        for c in range(int(off[u]), int(off[u + 1]), CHUNK):
            r = slice(c, min(c + CHUNK, int(off[u + 1])))
            e, w = err[r].norm(dim=(0, 2)), want[r].norm(dim=(0, 2))
            assert torch.all(e <= 2.0 ** -7 * w + 1e-30), (what, u, c, (e / w).tolist())


def near_long(got, want, mass, what=""):
    """`near` for tensors."""
    over = (got.double() - want).abs() - 2.0 ** -8 * want.abs() - (2.0 ** -8 + 2.0 ** -12) * mass - 1e-37
    assert torch.all(over <= 0), (what, int(over.argmax()), float(over.max()))
