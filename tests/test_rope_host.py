"""Rotary positions on the host: frequencies, the handle, refusals (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B
from broadcast_gemm_attention_gb300 import build
from qcache_util import rope_ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def test_frequencies_follow_their_definitions():
    rot, base = 16, 10000.0
    plain = np.array([base ** (-2 * j / rot) for j in range(8)])
    np.testing.assert_allclose(B.ikbo_rope_frequencies(rot), plain, rtol=1e-15)
    np.testing.assert_allclose(B.ikbo_rope_frequencies(rot, scaling="linear", factor=4.0), plain / 4, rtol=1e-15)
    wide = np.array([(base * 4.0 ** (16 / 14)) ** (-2 * j / rot) for j in range(8)])
    np.testing.assert_allclose(B.ikbo_rope_frequencies(rot, scaling="base", factor=4.0), wide, rtol=1e-14)
    got = np.array(B.ikbo_rope_frequencies(rot, scaling="turns", factor=8.0, original_len=8192.0, low_turns=1.0,
                                           high_turns=4.0))
    turns = 8192.0 * plain / (2 * math.pi)
    assert (turns >= 4).any() and (turns <= 1).any() and ((turns > 1) & (turns < 4)).any()
    np.testing.assert_allclose(got[turns >= 4], plain[turns >= 4], rtol=1e-15)
    np.testing.assert_allclose(got[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    keep = (turns[mid] - 1) / 3
    np.testing.assert_allclose(got[mid], plain[mid] * (keep + (1 - keep) / 8), rtol=1e-14)


def test_the_smallest_rotation():
    assert B.ikbo_rope_frequencies(2, scaling="base", factor=9.0) == [1.0]
    B.Rope(2)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=514), dict(base=0.0),
                                dict(base=math.inf), dict(factor=0.0), dict(factor=math.nan),
                                dict(scaling="turns", original_len=0.0), dict(scaling="turns", low_turns=2.0),
                                dict(scaling="turns", low_turns=-1.0), dict(scaling="turns", high_turns=math.inf)])
def test_frequencies_refuse(kw):
    args = dict(rot_dim=16, original_len=100.0)
    args.update(kw)
    with pytest.raises(B.IkboError) as e:
        B.ikbo_rope_frequencies(**args)
    assert e.value.code == B.IKBO_ERR_INVALID_ARG


def test_unknown_scaling_and_wrong_table_size():
    with pytest.raises(ValueError):
        B.ikbo_rope_frequencies(16, scaling="other")
    with pytest.raises(ValueError):
        B.Rope(16, [1.0] * 7)


@pytest.mark.parametrize("freqs,magnitude", [([math.nan], 1.0), ([math.inf], 1.0), ([1.0], 0.0), ([1.0], math.inf)])
def test_create_refuses(freqs, magnitude):
    with pytest.raises(B.IkboError) as e:
        B.Rope(2, freqs, magnitude=magnitude)
    assert e.value.code == B.IKBO_ERR_INVALID_ARG


def test_create_null_and_destroy_null():
    L = B.load()
    assert L.ikbo_rope_create(None, 2, None, 0, 1.0) == B.IKBO_ERR_INVALID_ARG
    h = ctypes.c_void_p(1)
    assert L.ikbo_rope_create(ctypes.byref(h), 2, None, 0, 1.0) == B.IKBO_ERR_INVALID_ARG
    assert h.value is None
    L.ikbo_rope_destroy(None)


def test_calls_refuse_before_any_launch():
    """Sizes and pointers are looked at before the plan, so a null plan shows what they say."""
    L, r = B.load(), B.Rope(16)
    strides = (ctypes.c_int64 * 3)(64, 16, 16)
    sp = ctypes.addressof(strides)
    ok = dict(plan=None, rope=r.handle, X=0x1000, xs=None, Y=0x2000, ys=None, start=None, broadcast=0, dtype=0, n=4,
              H=1, L=1, d=16, stream=None)
    for name in ("ikbo_rope_forward", "ikbo_rope_backward"):
        def call(**kw):
            a = dict(ok)
            a.update(kw)
            return getattr(L, name)(*a.values())
        invalid = [{}, dict(rope=None), dict(X=None), dict(Y=None), dict(n=-1), dict(H=0), dict(L=0), dict(d=0),
                   dict(dtype=3), dict(dtype=-1), dict(X=0x1001), dict(dtype=2, Y=0x2002), dict(start=0x3002),
                   dict(d=14), dict(Y=0x1000, ys=sp)]
        for kw in invalid:
            assert call(**kw) == B.IKBO_ERR_INVALID_ARG, kw
        assert call(d=514) == B.IKBO_ERR_UNSUPPORTED
        assert call(n=1 << 20, L=1 << 12) == B.IKBO_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 1, 1, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.ikbo_rope_forward(0, 0, x, x)


def test_the_reference_is_a_rotation():
    """The tests' own reference: closed forms."""
    x = np.zeros((1, 1, 2, 4))
    x[0, 0, :, 0] = 1.0
    y = rope_ref(x, np.array([[0, 1]]), [math.pi / 2, 0.3])
    np.testing.assert_allclose(y[0, 0, 0], [1, 0, 0, 0], atol=1e-15)
    np.testing.assert_allclose(y[0, 0, 1], [0, 0, 1, 0], atol=1e-15)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 4, 8))
    pos = rng.integers(-9, 1000000, (2, 4))
    f = [1.0, 0.1, 0.01]
    for inter in (False, True):
        y = rope_ref(x, pos, f, inter)
        np.testing.assert_allclose(rope_ref(y, pos, f, inter, backward=True), x, atol=1e-12)
        np.testing.assert_allclose((y ** 2).sum(), (x ** 2).sum(), rtol=1e-13)
