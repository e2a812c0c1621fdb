"""Bounds of every element of what linear attention computes, beside linattn_util (not collected by pytest).

An output in bf16 is a sum of terms (q.k decayed) v and q S.  On its way a term is rounded to bf16 once, its
product q.k with the decay or the state's element, by at most 2^-8 of its magnitude; the output is rounded
once, by 2^-8 of itself.  What else there is to it is small beside that: the state's own 2^-14 of its magnitudes
(test_gpu_linattn.py derives it) and fp32 sums of at most 256 terms, 2^-16.  With `mass` the sum of the terms'
magnitudes (the definition on absolute values), an element is off by at most
    2^-8 |o| + (2^-8 + 2^-8 2^-8 + 2^-14 + 2^-16) mass  <  2^-8 |o| + (2^-8 + 2^-12) mass,
where the third part of the middle bracket is the output's rounding of the first error."""
import numpy as np

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
