"""The long reference of linear attention's tests against the one row by row."""
import numpy as np
import torch

import linattn_bounds as BD
import linattn_util as R


def test_the_long_reference_is_the_definition(monkeypatch):
    monkeypatch.setattr(R, "D", 5)
    monkeypatch.setattr(BD, "CHUNK", 4)
    rng = np.random.default_rng(1)
    H, off, decay = 4, [0, 3, 3, 16, 20], np.array([0.9, 0.0, 1.0, 0.5])
    Q, K, V, dO = rng.standard_normal((4, 21, H, 5))
    S0, dS = rng.standard_normal((2, 4, H, 5, 5))
    t = torch.from_numpy
    for s, e in ((S0, dS), (None, None)):
        ts, te = (None if x is None else t(x) for x in (s, e))
        O, S, _ = BD.long_forward(t(Q), t(K), t(V), t(decay), off, ts, 0.7)
        O2, S2 = R.forward(Q, K, V, decay, off, s, 0.7)
        np.testing.assert_allclose(O, O2, atol=1e-12)
        np.testing.assert_allclose(S, S2, atol=1e-12)
        _, S, _ = BD.long_forward(None, t(K), t(V), t(decay), off, ts, 0.7)
        np.testing.assert_allclose(S, S2, atol=1e-12)
        for got, want in zip(BD.long_backward(t(Q), t(K), t(V), t(dO), t(decay), off, ts, te, 0.7), R.backward(Q, K, V, dO, decay, off, s, e, 0.7)):
            np.testing.assert_allclose(got, want, atol=1e-12)
