"""Memory that a plan holds for the cache attention: what its largest call needs,
not what all the calls before needed."""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import bf, i32
from test_gpu_qcache_attn import check, queries

pytestmark = pytest.mark.gpu

GIB = 2**30


class Decoded:
    """A request whose histories are decoded into the plan's workspace: 512 bytes for each of 8 heads
    and each token of the bound Lkv, whatever the lengths."""

    def __init__(self):
        self.st = R.Store(3, [90, 260], 8, 16)
        self.m = np.repeat(np.arange(2), 9).astype(np.int32)
        self.Q = queries(4, 18, 8, 128)
        self.q, self.cache = bf(self.Q), self.st.cuda()
        self.O = torch.zeros_like(self.q)

    def attend(self, p, tokens):
        data, table, lens = self.cache
        p.attn_qcache_forward(self.q, data, 16, table, lens, self.O, Lkv=tokens)

    def check(self):
        check(self.O, None, self.Q, self.st.kv, self.m, 8)


def used(before):
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


def test_a_growing_bound_keeps_one_workspace():
    r = Decoded()
    with B.Plan(18, 2, 8) as p:
        p.plan(i32(r.m), 2, 8, 128)
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        tokens = 60_000
        while tokens < 800_000:  # to 3 GiB
            r.attend(p, tokens)
            assert p.status() == B.IKBO_OK
            assert used(before) <= 1.26 * 4096 * (tokens + 256) + 2**26
            tokens = tokens * 13 // 10
        r.check()
        # a quarter more than this one would be above the largest there is, 8 GiB
        for gib in (6.6, 6.7):
            r.O.zero_()
            r.attend(p, int(gib * GIB / 4096))
        assert p.status() == B.IKBO_OK
        assert used(before) <= 8 * GIB + 2**26
        r.check()


def test_only_captured_workspaces_are_kept():
    """A graph's buffer outlives the calls that outgrow it, and later ones go when they are replaced."""
    r = Decoded()
    with B.Plan(18, 2, 8) as p:
        p.plan(i32(r.m), 2, 8, 128)
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        r.attend(p, 100_000)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r.attend(p, 100_000)
        held = used(before)  # with whatever the graph itself takes
        for tokens in (130_000, 170_000, 220_000, 290_000):
            r.attend(p, tokens)
            assert used(before) <= held + 1.26 * 4096 * (tokens + 256) + 2**26
        assert p.status() == B.IKBO_OK
        r.O.zero_()
        graph.replay()
        assert p.status() == B.IKBO_OK
        r.check()
        del graph


def test_a_plan_holds_less_after_it_is_destroyed():
    r = Decoded()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    with B.Plan(18, 2, 8) as p:
        p.plan(i32(r.m), 2, 8, 128)
        for tokens in (100_000, 200_000):
            r.attend(p, tokens)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                r.attend(p, tokens)
            del graph
    assert used(before) < 2**28
