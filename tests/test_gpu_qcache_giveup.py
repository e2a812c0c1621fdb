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
        self.Q = [queries(3 + k, self.m.size, 2, 8) for k in range(2)]
        self.q, self.cache = [bf(x) for x in self.Q], self.st.cuda()

    def plan(self, stream=None):
        p = B.Plan(self.m.size, 3, 2)
        p.plan(i32(self.m), 3, 2, 8, stream=stream)
        return p

    def attend(self, p, stream=None, k=0):
        """With the k-th queries."""
        data, table, lens = self.cache
        O = torch.zeros_like(self.q[k])
        if stream is not None:
            torch.cuda.synchronize()
        # so large a bound that this is not a few short histories: the tile kernel
        p.attn_qcache_forward(self.q[k], data, 64, table, lens, O, Lkv=8_000_000, stream=stream)
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
        check(before, None, r.Q[0], r.st.kv, r.m, 2)
        for _ in range(3):
            give_up(p, r)
            assert p.status() == B.IKBO_ERR_TIMEOUT
            assert torch.equal(r.attend(p), before)
            assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("side", [False, True])
def test_the_next_call_needs_no_status_read(side):
    """Every split's pieces are counted also where their CTA gave up: the calls after are
    right, on whichever stream, although nobody has read the status in between."""
    r = Request()
    stream = torch.cuda.Stream() if side else None
    with r.plan(stream) as p:
        before = [r.attend(p, stream, k) for k in range(2)]
        assert p.status(stream) == B.IKBO_OK
        for k in range(2):
            check(before[k], None, r.Q[k], r.st.kv, r.m, 2)
        for _ in range(3):
            give_up(p, r, stream)
            after = [r.attend(p, stream, k) for k in (1, 0, 1)]  # other rows than the ones that lie in the slots
            assert p.status(stream) == B.IKBO_ERR_TIMEOUT
            assert torch.equal(after[0], before[1]) and torch.equal(after[1], before[0]) and torch.equal(after[2], before[1])
        last = r.attend(p, stream)
        assert p.status(stream) == B.IKBO_OK
        assert torch.equal(last, before[0])
