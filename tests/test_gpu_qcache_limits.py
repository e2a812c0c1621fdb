"""Attention over the cache at the limits of its arguments: as many users as a plan
can have, and bounds on the tokens above 31 bits."""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import i32
from test_gpu_qcache_attn import attend, check, queries

pytestmark = pytest.mark.gpu

USERS = 8192


@pytest.fixture(scope="module")
def store():
    lens = np.random.default_rng(8).integers(0, 4, USERS)
    lens[[0, 5000]] = 300, 700
    return R.Store(8, lens.tolist(), 1, 16)


@pytest.mark.parametrize("n,Lq,Lkv", [
    (100, 8, None),          # in registers, a CTA an item
    (USERS, 8, None),        # a warp an item, 8 rows
    (USERS, 16, None),       # 16 rows
    (3 * USERS, 8, 2**24),   # in tiles
    (200, 8, 2**31 - 1),
])
def test_most_users(store, n, Lq, Lkv):
    rng = np.random.default_rng(n)
    m = rng.integers(0, USERS, n).astype(np.int32) if n < USERS else np.tile(np.arange(USERS), n // USERS).astype(np.int32)
    m[:3] = 0, 5000, USERS - 1
    m = rng.permutation(m)
    Q = np.tile(queries(5, 100, 1, Lq), (-(-n // 100), 1, 1, 1))[:n]
    with B.Plan(n, USERS, 1) as p:
        p.plan(i32(m), USERS, 1, Lq)
        O, lse = attend(p, Q, store, Lkv=Lkv or int(store.lens.sum()))
        assert p.status() == B.IKBO_OK
        again, _ = attend(p, Q, store, lse=False, Lkv=Lkv or int(store.lens.sum()))
        assert torch.equal(O, again) and not bool(torch.isnan(O).any())
        some = np.flatnonzero((m % 97 == 0) | (m == 5000) | (m == USERS - 1))
        check(O[some], lse[some], Q[some], store.kv, m[some], 1)


@pytest.mark.parametrize("bound", [2**31, 2**32 + 5, 2**40])
def test_a_bound_of_more_than_31_bits(bound):
    """Any bound is allowed: more than a cache can hold is the same as what it can hold."""
    st = R.Store(9, [40, 20], 1, 16)
    m = np.array([0, 1, 1], np.int32)
    Q = queries(6, 3, 1, 8)
    with B.Plan(3, 2, 1) as p:
        p.plan(i32(m), 2, 1, 8)
        O, lse = attend(p, Q, st, Lkv=bound)
        assert p.status() == B.IKBO_OK
        check(O, lse, Q, st.kv, m, 1)
