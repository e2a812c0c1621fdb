"""Attention over the cache in registers where every warp works alone: hundreds of
users with a row or two of queries each, in tiles of 8 and of 16 rows."""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import i32
from test_gpu_qcache_attn import attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,H_kv,Lq", [(8, 8, 8), (8, 8, 16), (16, 8, 8)])
@pytest.mark.parametrize("outside", [False, True])
def test_a_warp_an_item(H, H_kv, Lq, outside):
    """500 users of 8 rows (or 16) over 8 K/V heads: an item and more for every warp.  One
    history is cut over many of them, some are empty, one user has a tenth of the candidates."""
    users = 500
    rng = np.random.default_rng(H + Lq)
    lens = rng.integers(0, 40, users)
    lens[[1, users - 1]] = 0, 1
    lens[users // 2] = 4000
    st = R.Store(users, lens.tolist(), H_kv, 16)
    m = np.arange(users)
    m[rng.random(users) < 0.1] = users // 2
    m = rng.permutation(m).astype(np.int32)
    if outside:
        m[rng.random(users) < 0.05] = users
    Q = np.tile(queries(4, 50, H, Lq), (10, 1, 1, 1))
    with B.Plan(users, users, H) as p:
        p.plan(i32(m), users, H, Lq)
        O, lse = attend(p, Q, st, Lkv=int(lens.sum()))
        assert p.status() == (B.IKBO_ERR_MAP_OUT_OF_RANGE if outside else B.IKBO_OK)
        assert torch.equal(torch.isnan(O).flatten(1).any(1).cpu(), torch.from_numpy(m == users))
        for _ in range(3):
            again, _ = attend(p, Q, st, lse=False, Lkv=int(lens.sum()))
            assert torch.equal(O[torch.from_numpy(m < users)], again[torch.from_numpy(m < users)])
        some = np.flatnonzero((m % 13 == 0) | (m == users - 1) | (m == 1))
        some = np.concatenate([some, np.flatnonzero(m == users // 2)[:6]])
        check(O[some], lse[some], Q[some], st.kv, m[some], H_kv)
