"""The cache attention's tile kernel when a wait inside it runs out.

A debug switch keeps every fourth CTA's keys from the products; the waits for
them end at the plan's limit, the call reports it, and nothing of it is
left for the calls after.  (A wait that looks at its limit every 64 tries takes
longer than the limit asked for, but ends.)
"""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import bf, i32
from test_gpu_qcache_attn import check, queries

pytestmark = pytest.mark.gpu


class Request:
    """Three histories whose tiles are split over CTAs, two with rows for all of a tile's warps."""

    def __init__(self):
        self.st = R.Store(1, [2500, 1900, 3300], 2, 64)
        self.m = np.repeat(np.arange(3), [16, 3, 40]).astype(np.int32)
        self.Q = queries(3, self.m.size, 2, 8)
        self.q, self.cache = bf(self.Q), self.st.cuda()

    def plan(self, stream=None):
        p = B.Plan(self.m.size, 3, 2)
        p.plan(i32(self.m), 3, 2, 8, stream=stream)
        return p

    def attend(self, p, stream=None):
        data, table, lens = self.cache
        O = torch.zeros_like(self.q)
        if stream is not None:
            torch.cuda.synchronize()
        # so large a bound that this is not a few short histories: the tile kernel
        p.attn_qcache_forward(self.q, data, 64, table, lens, O, Lkv=8_000_000, stream=stream)
        return O


def give_up(p, r, stream=None):
    """One call whose waits run out."""
    B.ikbo_plan_set_timeout_ns(p.handle, 5_000_000)
    B.ikbo_plan_set_debug(p.handle, B.DEBUG_WITHHOLD_KEYS)
    r.attend(p, stream)
    B.ikbo_plan_set_debug(p.handle, 0)
    B.ikbo_plan_set_timeout_ns(p.handle, 2_000_000_000)


def test_a_wait_that_ran_out_is_reported_and_over():
    r = Request()
    with r.plan() as p:
        before = r.attend(p)
        assert p.status() == B.IKBO_OK
        check(before, None, r.Q, r.st.kv, r.m, 2)
        for _ in range(3):
            give_up(p, r)
            assert p.status() == B.IKBO_ERR_TIMEOUT
            assert torch.equal(r.attend(p), before)
            assert p.status() == B.IKBO_OK
