"""Linear attention, drafted trees and rotations with axes without a GPU: refusals, and
the tests' own references against differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import linattn_util as R
from broadcast_gemm_attention_gb300 import binding as B
from broadcast_gemm_attention_gb300 import build

INVALID, UNSUPPORTED = 1, 2
A = 0x10000  # an aligned address that is never used


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def _refusals(name, ok, invalid, unsupported):
    f = getattr(B.load(), name)
    for kws, code in ((invalid, INVALID), (unsupported, UNSUPPORTED)):
        for kw in kws:
            a = dict(ok)
            a.update(kw)
            assert f(*a.values()) == code, (name, kw)


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def test_forward_refuses():
    ok = dict(plan=None, Q=A, K=A + 16, V=A + 32, strides=None, off=A, n_users=4, n_rows=10, max_len=0, H=8, d=128, decay=A, s_in=A,
              s_out=A, O=A + 48, scale=1.0, stream=None)
    _refusals("ikbo_linattn_forward", ok,
              [{}] + [{k: None} for k in ("Q", "K", "V", "O", "decay")] + [{k: A + 8} for k in ("Q", "K", "V", "O", "s_in", "s_out")] +
              [dict(off=A + 2), dict(decay=A + 2), dict(n_users=0), dict(n_rows=-1), dict(max_len=-1), dict(H=0), dict(scale=0.0),
               dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e-40), dict(off=None), dict(O=A), dict(O=A + 16), dict(O=A + 32),
               dict(Q=None, O=None, s_out=None), dict(strides=strides(1016, 1024, 1024, 1024)),
               dict(strides=strides(1024, 1024, 1024, 512))],
              [dict(d=64), dict(n_users=8193), dict(H=1025), dict(strides=strides(1024, 1028, 1024, 1024))])


def test_backward_refuses():
    ok = dict(plan=None, Q=A, K=A + 16, V=A + 32, dO=A + 48, strides=None, off=A, n_users=4, n_rows=10, max_len=0, H=8, d=128,
              decay=A, s_in=A + 64, ds_out=A + 80, dQ=A + 96, dK=A + 112, dV=A + 128, ds_in=A + 144, scale=1.0, stream=None)
    _refusals("ikbo_linattn_backward", ok,
              [{}] + [{k: None} for k in ("Q", "K", "V", "dO", "decay")] +
              [{k: A + 8} for k in ("Q", "K", "V", "dO", "dQ", "dK", "dV", "s_in", "ds_out", "ds_in")] +
              [dict(dQ=None, dK=None, dV=None, ds_in=None), dict(dQ=A), dict(dK=A + 16), dict(dV=A + 48), dict(ds_in=A + 80),
               dict(ds_in=A + 64), dict(n_users=0), dict(scale=-1.0), dict(off=None),
               dict(strides=strides(1024, 1024, 1024, 1024, 1024, 1024, 8))],
              [dict(d=256), dict(n_users=9000), dict(strides=strides(1024, 1024, 1024, 1024, 1026, 1024, 1024))])


def test_reads_refuse():
    ok = dict(plan=None, Q=A, state=A, O=A, d=128, scale=1.0, stream=None)
    _refusals("ikbo_linattn_read_forward", ok,
              [{}] + [{k: None} for k in ("Q", "state", "O")] + [{k: A + 4} for k in ("Q", "state", "O")] +
              [dict(scale=0.0), dict(scale=math.nan)], [dict(d=64)])
    ok = dict(plan=None, Q=A, state=A, dO=A + 16, dQ=A + 32, ds=A + 48, d=128, scale=1.0, stream=None)
    _refusals("ikbo_linattn_read_backward", ok,
              [{}] + [{k: None} for k in ("Q", "state", "dO")] + [{k: A + 4} for k in ("Q", "state", "dO", "dQ", "ds")] +
              [dict(dQ=None, ds=None), dict(dQ=A), dict(dQ=A + 16), dict(ds=A), dict(scale=-2.0)], [dict(d=32)])


def test_tree_refuses():
    ok = dict(plan=None, Q=A, data=A, n_pages=10, page=64, H_kv=8, table=A, max_blocks=3, lens=A, K=A, V=A, stride=1024, parents=A,
              O=A + 16, lse=None, Lkv=10, d=128, scale=1.0, stream=None)
    _refusals("ikbo_attn_qcache_tree_forward", ok,
              [{}] + [{k: None} for k in ("Q", "data", "table", "lens", "K", "V", "O")] +
              [dict(Q=A + 8), dict(O=A), dict(O=A + 2), dict(K=A + 8), dict(V=A + 4), dict(parents=A + 2), dict(lse=A + 2), dict(Lkv=0),
               dict(scale=0.0), dict(H_kv=0), dict(stride=1016)],
              [dict(d=64), dict(page=17), dict(stride=1028)])


def test_rotations_with_axes_refuse():
    with pytest.raises(B.IkboError) as e:
        B.Rope(16, axes=[0, 1, 2, 3, 4, 0, 0, 0])  # five axes
    assert e.value.code == UNSUPPORTED
    with pytest.raises(B.IkboError):
        B.Rope(16, axes=[0, 1, 2, 0, 0, 0, 0, 0], n_axes=2)  # a pair on the third
    for bad in ([0] * 7, [-1] * 8, [300] * 8):
        with pytest.raises(ValueError):
            B.Rope(16, axes=bad)
    h = ctypes.c_void_p(5)
    assert B.load().ikbo_rope_create_axes(ctypes.byref(h), 16, None, 1, None, 0, 1.0) == INVALID and h.value is None
    assert B.load().ikbo_rope_create_axes(None, 16, None, 1, None, 0, 1.0) == INVALID
    plain, axes = B.Rope(16), B.Rope(16, axes=[0, 1] * 4, n_axes=3)
    assert axes.axes == 3 and plain.axes == 0
    # each kind of rotation is for its own calls (checked before anything else)
    args = (A, None, A, None, None)
    assert B.load().ikbo_rope_forward(None, axes.handle, *args, 0, 0, 1, 1, 1, 16, None) == INVALID
    assert B.load().ikbo_rope_axes_forward(None, plain.handle, *args, None, 0, 0, 0, 1, 1, 1, 16, None) == INVALID
    assert B.load().ikbo_rope_axes_backward(None, axes.handle, *args, A + 2, 0, 0, 0, 1, 1, 1, 16, None) == INVALID
    assert B.load().ikbo_rope_axes_backward(None, axes.handle, *args, A, -1, 0, 0, 1, 1, 1, 16, None) == INVALID
    assert B.load().ikbo_rope_axes_backward(None, axes.handle, *args, A, 3, 0, 0, 1, 1, 1, 16, None) == INVALID  # no plan


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        B.ikbo_linattn_forward(0, x, x, x, torch.ones(2), x, n_users=1)


def test_the_reference_gradient_is_the_forward_s(monkeypatch):
    """Differences of the plain forward along random directions, in a small head."""
    monkeypatch.setattr(R, "D", 5)
    rng = np.random.default_rng(0)
    H, off, scale = 2, [0, 3, 3, 7], 0.7
    decay = [0.9, 0.25]
    X = {k: rng.standard_normal((7, H, 5)) for k in ("Q", "K", "V")}
    S0, dS, dO = rng.standard_normal((3, H, 5, 5)), rng.standard_normal((3, H, 5, 5)), rng.standard_normal((7, H, 5))

    def loss(X, S0):
        O, S = R.forward(X["Q"], X["K"], X["V"], decay, off, S0, scale)
        return (O * dO).sum() + (S * dS).sum()

    dQ, dK, dV, dS0 = R.backward(X["Q"], X["K"], X["V"], dO, decay, off, S0, dS, scale)
    for name, grad in (("Q", dQ), ("K", dK), ("V", dV), ("S", dS0)):
        step = rng.standard_normal(grad.shape)
        at = lambda e: (loss(X, S0 + e * step) if name == "S" else loss(dict(X, **{name: X[name] + e * step}), S0))  # noqa: E731
        # the loss is a polynomial of degree one in each argument: a central difference is exact but for rounding
        np.testing.assert_allclose((at(1e-3) - at(-1e-3)) / 2e-3, (grad * step).sum(), rtol=1e-9)


def test_the_reference_tree():
    m = R.sees([-1, 0, 0, 1, -2, 4, 9, 3, -1])
    assert m[3].nonzero()[0].tolist() == [0, 1, 3] and m[7].nonzero()[0].tolist() == [0, 1, 3, 7]
    assert m[2].nonzero()[0].tolist() == [0, 2] and m[8].nonzero()[0].tolist() == [8]
    assert not m[4].any() and not m[5].any() and not m[6].any()
