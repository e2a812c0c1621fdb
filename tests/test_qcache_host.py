"""The 4-bit cache without a GPU: refusals, sizes, and the tests' own references."""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from broadcast_gemm_attention_gb300 import build

INVALID, UNSUPPORTED = 1, 2
A = 0x10000  # an aligned address that is never used


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def test_bytes():
    assert B.ikbo_qcache_bytes(10, 64, 8) == 10 * 8 * 4 * 2560
    assert B.ikbo_qcache_bytes(1, 16, 1) == 2560
    for bad in ((0, 16, 1), (1, 8, 1), (1, 48, 1), (1, 2048, 1), (1, 16, 0), (1 << 27, 16, 1)):
        assert B.ikbo_qcache_bytes(*bad) == 0, bad
    assert B.ikbo_qcache_bytes((1 << 27) - 1, 16, 8) == ((1 << 27) - 1) * 8 * 2560


def _refusals(name, ok, invalid, unsupported):
    f = getattr(B.load(), name)
    for kws, code in ((invalid, INVALID), (unsupported, UNSUPPORTED)):
        for kw in kws:
            a = dict(ok)
            a.update(kw)
            assert f(*a.values()) == code, (name, kw)


def test_resize_refuses():
    ok = dict(plan=None, lens=A, new=A, n_users=4, table=A, max_blocks=8, page=16, free=A, n_free=A, n_pages=100,
              slots=A, offsets=A, positions=None, max_new=10, stream=None)
    _refusals("ikbo_qcache_resize", ok,
              [{}] + [{k: None} for k in ("lens", "new", "table", "free", "n_free", "slots", "offsets")] +
              [{k: A + 2} for k in ("lens", "new", "table", "free", "n_free", "slots", "offsets", "positions")] +
              [dict(n_users=0), dict(max_blocks=0), dict(n_pages=0), dict(max_new=-1)],
              [dict(n_users=8193), dict(page=24), dict(page=8), dict(max_blocks=1 << 28), dict(n_pages=1 << 28)])


def test_append_refuses():
    ok = dict(plan=None, K=A, V=A, stride=1024, slots=A, n_rows=3, H=8, d=128, data=A, n_pages=10, page=64, stream=None)
    _refusals("ikbo_qcache_append", ok,
              [{}] + [{k: None} for k in ("K", "V", "slots", "data")] + [{k: A + 8} for k in ("K", "V", "data")] +
              [dict(slots=A + 1), dict(n_rows=-1), dict(H=0), dict(n_pages=0), dict(stride=1016)],
              [dict(d=64), dict(page=40), dict(stride=1028), dict(n_pages=1 << 26)])


def test_load_refuses():
    ok = dict(plan=None, data=A, n_pages=10, page=64, H=8, d=128, table=A, max_blocks=3, lens=A, n_users=4, off=A, K=A,
              V=A, n_rows=10, stream=None)
    _refusals("ikbo_qcache_load", ok,
              [{}] + [{k: None} for k in ("data", "table", "lens", "off")] +
              [dict(K=A + 8), dict(V=A + 4), dict(data=A + 8), dict(off=A + 1), dict(n_rows=-1), dict(n_users=0),
               dict(H=0), dict(max_blocks=0)],
              [dict(d=256), dict(page=0), dict(n_users=9000), dict(max_blocks=1 << 27)])


def test_attention_refuses():
    ok = dict(plan=None, Q=A, data=A, n_pages=10, page=64, H_kv=8, table=A, max_blocks=3, lens=A, O=A, lse=None, Lkv=10,
              d=128, scale=1.0, stream=None)
    _refusals("ikbo_attn_qcache_forward", ok,
              [{}] + [{k: None} for k in ("Q", "data", "table", "lens", "O")] +
              [dict(Q=A + 8), dict(O=A + 2), dict(data=A + 8), dict(lse=A + 2), dict(Lkv=0), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0), dict(H_kv=0), dict(max_blocks=0)],
              [dict(d=64), dict(page=17), dict(max_blocks=1 << 28), dict(n_pages=1 << 28)])


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    data = torch.zeros(1, 1, 1, 2560, dtype=torch.uint8)
    x = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.ikbo_qcache_append(0, x, x, i, data, 16)
    with pytest.raises(ValueError):
        B.ikbo_qcache_resize(0, i, i, i.view(2, 1), 16, i, i[:1], i, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.ikbo_qcache_load(0, data, 16, i.view(2, 1), i, i, x, x)
    with pytest.raises(ValueError):
        B.ikbo_attn_qcache_forward(0, x.view(2, 1, 1, 128), data, 16, i.view(2, 1), i, x.view(2, 1, 1, 128))


def test_status_names():
    for code in (B.IKBO_ERR_OUT_OF_PAGES, B.IKBO_ERR_CACHE):
        assert code in B.STATUS_NAMES and B.ikbo_status_string(code) != "unknown status"


# ------------------------------------------------------- the references
def test_quantising_keeps_values_within_a_step():
    """|value - x| <= s (1/2 for the rounding + 1/32 for z's, 15 * 2^-8 for s's) + 2^-8 |value|."""
    rng = np.random.default_rng(1)
    x = R.bf16(rng.standard_normal((200, 128)) * 10.0 ** rng.integers(-3, 4, (200, 1)) + rng.integers(-2, 3, (200, 1)))
    c, s, z = R.quantise(x)
    v = R.values(c, s, z)
    step = np.repeat(s, 32, axis=-1)
    # z's rounding: 2^-8 |z|, at most 2^-8 (|lo| + 16 s)
    off = 2.0 ** -8 * np.abs(np.repeat(z, 32, axis=-1))
    assert np.all(np.abs(v - x) <= step * (0.5 + 15 * 2.0 ** -8) + off + 2.0 ** -8 * np.abs(v))


def test_a_constant_group_reads_back_exactly():
    x = np.full((1, 128), 0.3, np.float32)
    x = R.bf16(x)
    assert np.array_equal(R.values(*R.quantise(x)), x)


def test_the_store_reads_what_it_wrote():
    st = R.Store(3, [5, 0, 40], 2, 16)
    assert [len(k) for k, _ in st.kv] == [5, 0, 40]
    assert all(np.isfinite(k).all() and np.isfinite(v).all() for k, v in st.kv)


def test_the_resize_reference_keeps_every_page_once():
    rng = np.random.default_rng(5)
    U, B_, page, n_pages = 6, 5, 16, 24
    lens, table = np.zeros(U, np.int32), np.full((U, B_), -1, np.int32)
    free, n_free = rng.permutation(n_pages).astype(np.int32), n_pages
    for _ in range(40):
        new = rng.integers(0, B_ * page + 1, U)
        ok, lens, table, free, n_free, slots, off, pos = R.resize(lens, new, table, page, free, n_free, 600)
        held = sorted([int(x) for x in table.ravel() if x >= 0] + [int(x) for x in free[:n_free]])
        assert held == list(range(n_pages))
        assert len(set(slots[slots >= 0].tolist())) == int((slots >= 0).sum()) == off[-1]
