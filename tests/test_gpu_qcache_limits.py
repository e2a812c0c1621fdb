"""Attention over the cache at the limits of its arguments: as many users as a plan
can have, bounds on the tokens above 31 bits, and scores of any documented size."""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import i32
from test_gpu_qcache_attn import VARIANTS, attend, check, queries

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


@pytest.mark.parametrize("variant,exponents", [("registers", (12, 20, 23, 26)), ("tiles", (12, 20, 23, 26)), ("decoded", (12, 20))])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(variant, exponents, sign):
    """Scores of one sign, up to 2^26 (2^21 where histories are decoded first), of which one key's is the
    largest by far (by 2^-6 of itself, at least 16): its value is the result, to the bit but for P's part of
    the sum (e^-16)."""
    c, Lq, Lkv = VARIANTS[variant]["c"], VARIANTS[variant]["Lq"], VARIANTS[variant]["Lkv"]
    lens, best = [300, 700], [7, 512]
    st = R.Store(14, lens, 1, 16)
    m = np.repeat(np.arange(2), c).astype(np.int32)
    for e in exponents:
        for u in range(2):
            # keys along one coordinate: all sign 2^e / a, the best one less or more by 2^-6
            a = 2.0 ** (e // 2)
            k = np.zeros((lens[u], 1, 128), np.float32)
            k[:, 0, 0] = sign * 2.0 ** (e - e // 2)
            k[best[u], 0, 0] *= 1 + sign * 2.0 ** -6
            slots = [int(st.table[u, t // 16]) * 16 + t % 16 for t in range(lens[u])]
            R.store(st.data, 16, slots, R.bf16(k), st.kv[u][1])
        kv = [R.read(st.data, 16, st.table[u], lens[u]) for u in range(2)]
        Q = np.zeros((m.size, 1, Lq, 128), np.float32)
        Q[..., 0] = a
        with B.Plan(m.size, 2, 1) as p:
            p.plan(i32(m), 2, 1, Lq)
            O, lse = attend(p, Q, st, Lkv=Lkv, scale=1.0)
            assert p.status() == B.IKBO_OK
        O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
        for i, u in enumerate(m):
            K, V = kv[u]
            S = a * K[:, 0, 0].astype(np.float64)
            top = int(S.argmax())
            assert np.all(np.delete(S, top) <= S[top] - 16)
            v = V[top, 0].astype(np.float64)
            # P and the output in bf16 (2^-8 each), the other keys' part of the sum
            assert np.all(np.abs(O[i, 0] - v) <= 2.0 ** -7 * np.abs(v) + 700 * np.exp(-16) * 8), e
            assert np.all(np.abs(lse[i, 0] - S[top]) <= 2.0 ** -22 * abs(S[top]) + 1e-3)
