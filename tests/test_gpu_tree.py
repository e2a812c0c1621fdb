"""Attention of drafted trees over the 4-bit cache against the definition in 64 bits
(linattn_util.tree derives the bound of every element)."""
import math

import numpy as np
import pytest
import torch

import linattn_util as R
import qcache_util as QC
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import bf, i32

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


def draft(seed, n, Lq, branch=3, missing=True):
    rng = np.random.default_rng(seed)
    par = np.maximum(np.arange(Lq)[None, :] - rng.integers(1, branch + 1, (n, Lq)), -1)
    if missing:
        size = rng.integers(0, Lq + 1, (n, 1))
        size[0] = Lq
        par = np.where(np.arange(Lq)[None, :] < size, par, -2)
    return par.astype(np.int32)


class Case:
    def __init__(self, seed, lens, m, H, H_kv, Lq, page, parents=None, branch=3):
        rng = np.random.default_rng(seed)
        self.st = QC.Store(seed, lens, H_kv, page)
        self.m, self.H, self.H_kv, self.Lq = np.asarray(m, np.int32), H, H_kv, Lq
        n = len(m)
        self.Q = QC.bf16(rng.standard_normal((n, H, Lq, 128)))
        self.K, self.V = (QC.bf16(rng.standard_normal((n, Lq, H_kv, 128))) for _ in range(2))
        self.parents = draft(seed, n, Lq, branch) if parents is None else parents

    def run(self, p, lse=True, parents=True, Lkv=None, K=None, V=None, stream=None, O=None):
        data, table, ln = self.st.cuda()
        q = bf(self.Q)
        O = torch.full_like(q, float("nan")) if O is None else O
        L = torch.full(self.Q.shape[:3], float("nan"), device="cuda") if lse else None
        mm = i32(self.m)
        p.plan(mm, len(self.st.lens), self.H, self.Lq)
        if stream is not None:
            torch.cuda.synchronize()
        p.attn_qcache_tree_forward(q, data, self.st.page, table, ln, bf(self.K) if K is None else K, bf(self.V) if V is None else V,
                                   i32(self.parents) if parents else None, O, lse=L, Lkv=Lkv, stream=stream)
        return O, L

    def check(self, O, lse, parents=None):
        O64, l64, bound = R.tree(self.Q, self.st.kv, self.K, self.V, self.parents if parents is None else parents, self.m, self.H_kv, SCALE)
        inside = np.array([0 <= u < len(self.st.kv) for u in self.m])
        got = O.double().cpu().numpy()
        over = np.abs(got - O64) - bound
        assert np.all(over[inside] <= 0), float(np.nanmax(over[inside]))
        if lse is not None:
            g, w = lse.double().cpu().numpy()[inside], l64[inside]
            assert np.array_equal(np.isneginf(g), np.isneginf(w))
            fine = np.isfinite(w)
            assert np.all(np.abs(g[fine] - w[fine]) <= 1e-4 * (1 + np.abs(w[fine])))


def plan():
    return B.Plan(1024, 64, 16)


CASES = [
    # lens, map, H, H_kv, Lq, page
    ([1], [0], 1, 1, 8, 16),
    ([0], [0], 1, 1, 8, 16),
    ([33, 0, 17], [0, 1, 2, 0], 2, 2, 8, 16),
    ([1000], [0], 8, 8, 8, 64),
    ([70, 0, 128], [2, 2, 0, 1, 2], 4, 1, 16, 32),
    ([200, 5], [0, 1, 1], 6, 2, 24, 16),
    ([40], [0, 0], 2, 1, 40, 16),
    ([130, 64], [1, 0], 2, 2, 128, 128),
    ([20], [0], 8, 2, 128, 16),
    ([300, 1], [0] * 20 + [1] * 3, 3, 3, 16, 64),
]


@pytest.mark.parametrize("lens,m,H,H_kv,Lq,page", CASES)
def test_against_the_definition(lens, m, H, H_kv, Lq, page):
    c = Case(len(m) + Lq, lens, m, H, H_kv, Lq, page)
    with plan() as p:
        O, lse = c.run(p)
        c.check(O, lse)
        O2, _ = c.run(p, lse=False)
        c.check(O2, None)
        assert p.status() == B.IKBO_OK
        # the plan, the attention's launches and one more
        before = p.launches()
        c.run(p)
        assert p.launches() == before + 3


@pytest.mark.parametrize("Lkv", [8_000_000, 700])
def test_many_rows_a_user(Lkv):
    """The history's part in tiles and decoded first."""
    c = Case(5, [300], [0] * 10, 2, 1, 128, 64)
    with plan() as p:
        O, lse = c.run(p, Lkv=Lkv)
        c.check(O, lse)
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("Lq", [8, 72, 128])
def test_chains(Lq):
    """Without parents a draft is a chain; the deepest tree there is."""
    c = Case(6, [50, 0], [0, 1], 2, 1, Lq, 16)
    chain = np.tile(np.arange(-1, Lq - 1, dtype=np.int32), (2, 1))
    with plan() as p:
        O, lse = c.run(p, parents=False)
        c.check(O, lse, chain)
        c.parents = chain
        O2, lse2 = c.run(p)
        assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_many_roots_and_empty_drafts():
    Lq = 32
    par = np.full((3, Lq), -1, np.int32)
    par[1] = -2
    par[2, ::2] = -5
    c = Case(7, [40], [0, 0, 0], 2, 2, Lq, 16, parents=par)
    with plan() as p:
        O, lse = c.run(p)
        c.check(O, lse)
        assert not O[1].any() and torch.all(torch.isneginf(lse[1]))
        assert p.status() == B.IKBO_OK


def test_a_draft_is_its_rows_added_to_the_history():
    """A chain over a history reads what a candidate reads once the chain is stored (up to its rounding to 4 bits):
    with K and V that 4 bits hold exactly, the two agree within their bounds."""
    rng = np.random.default_rng(8)
    H, Lq, L = 2, 8, 37
    c = Case(8, [L], [0], H, H, Lq, 16, parents=np.arange(-1, Lq - 1, dtype=np.int32)[None])
    # rows that quantising gives back as they are
    for x in (c.K, c.V):
        x[...] = QC.values(*QC.quantise(x))
    c.Q[:] = c.Q[:, :, -1:]  # every row the same query: the last one reads all
    with plan() as p:
        O, lse = c.run(p)
        c.check(O, lse)
    full = [(np.concatenate([c.st.kv[0][k], x[0]])) for k, x in ((0, c.K), (1, c.V))]
    O64, _, bound = QC.attend(c.Q[:, :, -1:], [tuple(full)], [0], H, SCALE)
    assert np.all(np.abs(O[:, :, -1:].double().cpu().numpy() - O64) <= bound * 2)


@pytest.mark.parametrize("what", ["rows that are not there", "rows that no other reads"])
def test_infinities_and_nan_stay_where_they_are(what):
    Lq = 24
    par = np.full((2, Lq), -1, np.int32)
    par[:, 1:10] = np.arange(9)
    bad = [3] if what == "rows that are not there" else [12, 23]
    if what == "rows that are not there":
        par[:, 3] = -2
        par[:, 4:10] = -1
    c = Case(9, [20, 0], [0, 1], 4, 2, Lq, 16, parents=par)
    with plan() as p:
        ref, lref = c.run(p)
        K, V = bf(c.K), bf(c.V)
        for k, r in enumerate(bad):
            K[:, r] = float("nan")
            V[:, r] = float("inf") if k else float("nan")
            V[:, r, :, 5::7] = float("-inf")
        O, lse = c.run(p, K=K, V=V)
        others = [r for r in range(Lq) if r not in bad]
        assert torch.equal(O[:, :, others], ref[:, :, others]) and torch.equal(lse[:, :, others], lref[:, :, others])
        if what != "rows that are not there":
            assert torch.all(torch.isnan(O[:, :, bad]))
        # an infinite value that is read: infinite where it counts, and NaN nowhere
        V = bf(c.V)
        V[:, 0, :, 17] = float("inf")
        O, _ = c.run(p, V=V)
        if what == "rows that no other reads":
            assert torch.all(O[:, :, 0:10, 17] == float("inf")) and torch.equal(O[:, :, 10:], ref[:, :, 10:])
            assert torch.all(torch.isfinite(O[..., :17])) and torch.all(torch.isfinite(O[..., 18:]))


def test_bad_parents_are_reported():
    Lq = 16
    par = np.arange(-1, Lq - 1, dtype=np.int32)[None].repeat(3, 0)
    par[0, 5] = 5    # itself
    par[1, 2] = 900
    par[2, 7] = -2   # not there, but the row below it names it
    c = Case(10, [30], [0, 0, 0], 2, 2, Lq, 16, parents=par)
    with plan() as p:
        O, lse = c.run(p)
        assert p.status() == B.IKBO_ERR_CACHE
        c.check(O, lse)  # such rows, and those below them, are not there
        par[2] = -1
        par[0] = par[1] = -2
        c.run(p)
        assert p.status() == B.IKBO_OK


def test_a_candidate_out_of_range_keeps_its_rows():
    c = Case(11, [30], [0, 3, 0], 2, 2, 8, 16)
    with plan() as p:
        O = torch.full(c.Q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
        O, lse = c.run(p, O=O)
        c.check(O, lse)
        assert torch.all(O[1] == -7.0)
        assert p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE


def test_strided_rows_repeat_captured_and_on_another_stream():
    c = Case(12, [100, 60], [0, 1, 0], 4, 2, 16, 16)
    with plan() as p:
        O, lse = c.run(p)
        kv = torch.stack([bf(c.K), bf(c.V)], dim=2).contiguous()  # [n, Lq, 2, H_kv, 128]
        O2, lse2 = c.run(p, K=kv[:, :, 0], V=kv[:, :, 1])
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
        side = torch.cuda.Stream()
        O3, _ = c.run(p, lse=False, stream=side)
        side.synchronize()
        assert torch.equal(O, O3)
        data, table, ln = c.st.cuda()
        q, K, V, par, O4 = bf(c.Q), bf(c.K), bf(c.V), i32(c.parents), torch.zeros_like(O)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            p.attn_qcache_tree_forward(q, data, c.st.page, table, ln, K, V, par, O4)
        for _ in range(2):
            O4.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(O4, O)
        with pytest.raises(ValueError):
            p.attn_qcache_tree_forward(q, data, c.st.page, table, ln, K[:, :8], V[:, :8], par, O4)
        with pytest.raises(ValueError):
            p.attn_qcache_tree_forward(q, data, c.st.page, table, ln, K, V, par[:, :8], O4)
        assert p.status() == B.IKBO_OK


def test_inputs_that_change_right_before_and_after_a_call():
    """The drafts' part may be set up while the history's ends: not before what is ahead of the call, nor past what is behind it."""
    c, other = Case(14, [300, 90], [0, 1, 0, 1, 1], 4, 2, 16, 16), Case(15, [300, 90], [0, 1, 0, 1, 1], 4, 2, 16, 16)
    with plan() as p:
        other.st, other.Q = c.st, c.Q
        want = [(k, *k.run(p)) for k in (c, other)]
        data, table, ln = c.st.cuda()
        ins = [(bf(k.K), bf(k.V), i32(k.parents)) for k, _, _ in want]
        q, K, V, par = bf(c.Q), *(torch.zeros_like(t) for t in ins[0])
        O, lse = torch.zeros_like(q), torch.zeros_like(want[0][2])
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")

        def once(i):
            for to, x in zip((K, V, par), ins[i]):
                to.copy_(x)
            p.attn_qcache_tree_forward(q, data, c.st.page, table, ln, K, V, par, O, lse=lse)
            for to in (K, V, par):
                to.fill_(-1)
            wrong.add_((O != want[i][1]).sum() + (lse != want[i][2]).sum())
            O.zero_()
            lse.zero_()

        for i in range(100):
            once(i % 2)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            once(0)
            once(1)
        for _ in range(20):
            graph.replay()
        torch.cuda.synchronize()
        assert p.status() == B.IKBO_OK and int(wrong) == 0


@pytest.mark.parametrize("Lq,H,H_kv", [(24, 4, 4), (40, 8, 4), (56, 6, 1), (104, 4, 2)])
def test_long_drafts_whose_keys_are_shared(Lq, H, H_kv):
    """More CTAs than fit, rows that are slices of one projection, sizes that are no multiples of a block (Lq is a multiple of 8)."""
    rng = np.random.default_rng(Lq)
    m = rng.integers(0, 3, 90).astype(np.int32)
    c = Case(60 + Lq, [120, 0, 37], m, H, H_kv, Lq, 16, branch=5)
    with plan() as p:
        O, lse = c.run(p)
        c.check(O, lse)
        kv = torch.stack([bf(c.K), bf(c.V)], dim=2).contiguous()
        O2, lse2 = c.run(p, K=kv[:, :, 0], V=kv[:, :, 1])
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
        assert p.status() == B.IKBO_OK
