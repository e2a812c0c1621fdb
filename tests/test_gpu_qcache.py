"""The 4-bit cache on the GPU: lengths, pages and slots (exact), quantised
bytes (exact, to the definition's own roundings), histories read back."""
import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Tables:
    """lens, table, free list on both sides."""

    def __init__(self, U, max_blocks, page, n_pages, seed=0):
        self.page, self.n_pages = page, n_pages
        self.lens, self.table = np.zeros(U, np.int32), np.full((U, max_blocks), -1, np.int32)
        self.free, self.n_free = np.random.default_rng(seed).permutation(n_pages).astype(np.int32), n_pages
        self.dev = [i32(self.lens), i32(self.table), i32(self.free), i32([self.n_free])]

    def resize(self, p, new, max_new, positions=True):
        ok, self.lens, self.table, self.free, self.n_free, slots, off, pos = R.resize(
            self.lens, new, self.table, self.page, self.free, self.n_free, max_new)
        lens, table, free, n_free = self.dev
        s, q = (torch.full((max_new,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        o = torch.full((len(self.lens) + 1,), -7, dtype=torch.int32, device="cuda")
        p.qcache_resize(lens, i32(new), table, self.page, free, n_free, s, o, q if positions else None)
        for got, want, name in ((lens, self.lens, "lens"), (table, self.table, "table"), (free, self.free, "free"),
                                (s, slots, "slots"), (o, off, "offsets")):
            assert np.array_equal(got.cpu().numpy(), want), name
        assert n_free.item() == self.n_free
        if positions:
            assert np.array_equal(q.cpu().numpy(), pos)
        return ok, s, o, q


@pytest.mark.parametrize("U,page,max_blocks", [(1, 16, 1), (3, 16, 4), (33, 32, 7), (1000, 64, 3), (1025, 16, 5),
                                               (8192, 16, 2)])
def test_resize_follows_the_definition(U, page, max_blocks):
    rng = np.random.default_rng(U)
    t = Tables(U, max_blocks, page, max(1, U * max_blocks * 2 // 3), seed=U)
    seen = set()
    with B.Plan(1, 1) as p:
        for step in range(6):
            new = rng.integers(0, max_blocks * page + 1, U)
            if step == 0:
                new //= 2
            if step == 3:
                new = t.lens.copy()  # nothing changes
            if step == 4:
                new = np.zeros(U, np.int32)
            added = int(np.maximum(new - t.lens, 0).sum())
            ok, *_ = t.resize(p, new, added + (step % 2) * 5, positions=step != 1)
            st = p.status()
            assert st == (B.IKBO_OK if ok else B.IKBO_ERR_OUT_OF_PAGES)
            seen.add(ok)
    assert True in seen


def test_resize_with_many_tokens_uses_the_cluster():
    t = Tables(40, 40, 64, 1600, seed=9)
    rng = np.random.default_rng(3)
    with B.Plan(1, 1) as p:
        for _ in range(4):
            new = rng.integers(0, 2561, 40)
            t.resize(p, new, 102400)
            assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("new,lens,n_free,max_new", [([17, -1], None, None, 100), ([17, 65], None, None, 100),
                                                     ([17, 5], [0, 99], None, 100), ([17, 5], [-3, 0], None, 100),
                                                     ([17, 5], None, 99, 100), ([17, 5], None, -1, 100),
                                                     ([17, 5], None, None, 21), ([2**31 - 1, 2**31 - 1], None, None, 5)])
def test_resize_refuses_as_a_whole(new, lens, n_free, max_new):
    t = Tables(2, 4, 16, 8)
    if lens is not None:
        t.lens = np.array(lens, np.int32)
        t.dev[0] = i32(lens)
    if n_free is not None:
        t.n_free = n_free
        t.dev[3] = i32([n_free])
    with B.Plan(1, 1) as p:
        ok, *_ = t.resize(p, new, max_new)
        assert not ok and p.status() == B.IKBO_ERR_CACHE
        assert p.status() == B.IKBO_OK  # reported once


def test_resize_reports_broken_pages():
    """A page number out of range in the free list or the table: reported, and its tokens have no slot."""
    with B.Plan(1, 1) as p:
        t = Tables(1, 4, 16, 8)
        t.dev[2][:] = 50
        lens, table, free, n_free = t.dev
        s, o = i32([0] * 20), i32([0, 0])
        p.qcache_resize(lens, i32([20]), table, 16, free, n_free, s, o)
        assert p.status() == B.IKBO_ERR_CACHE
        assert bool((s == -1).all())


def test_resize_of_no_tokens_and_in_a_graph():
    t = Tables(4, 8, 16, 32)
    lens, table, free, n_free = t.dev
    new, slots, off = i32([30, 0, 7, 128]), i32([0] * 165), i32([0] * 5)
    with B.Plan(1, 1) as p:
        p.qcache_resize(lens, i32([0] * 4), table, 16, free, n_free, slots[:0], off)
        assert off.tolist() == [0] * 5
        keep = [x.clone() for x in t.dev]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.qcache_resize(lens, new, table, 16, free, n_free, slots, off)
        for x, k in zip(t.dev, keep):
            assert torch.equal(x, k)  # captured, not run
        graph.replay()
        ok, l2, t2, f2, nf2, s2, o2, _ = R.resize([0] * 4, [30, 0, 7, 128], t.table, 16, t.free, t.n_free, 165)
        assert ok and np.array_equal(slots.cpu().numpy(), s2) and np.array_equal(table.cpu().numpy(), t2)
        assert n_free.item() == nf2 and p.status() == B.IKBO_OK


# ---------------------------------------------------------------- append
def rows(seed, n, H):
    """Rows of every kind: ordinary, constant, tiny, huge, one-sided, signed zeros, infinities, NaN."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, H, 128)).astype(np.float32)
    kinds = rng.integers(0, 10, n)
    for r in range(n):
        k = kinds[r]
        if k == 1:
            x[r] = x[r, :, :1]
        elif k == 2:
            x[r] *= np.float32(1e-38)
        elif k == 3:
            x[r] *= np.float32(1e37)
        elif k == 4:
            x[r] = np.abs(x[r]) + 100
        elif k == 5:
            x[r] = np.where(x[r] > 0, np.float32(0), np.float32(-0.0))
        elif k == 6:
            x[r, 0, 17] = np.inf
        elif k == 7:
            x[r, -1, 127] = np.nan
        elif k == 8:
            x[r, 0, 64] = np.float32(3e38)
            x[r, 0, 65] = np.float32(-3e38)
        elif k == 9:
            x[r] = rng.integers(-8, 8, x[r].shape)  # many exact ties
    return R.bf16(x)


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("n,H,page", [(1, 1, 16), (7, 3, 16), (50, 8, 32), (300, 2, 64), (129, 5, 1024)])
def test_append_writes_the_defined_bytes(n, H, page):
    n_pages = n // page + 5
    rng = np.random.default_rng(n)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    slots[rng.random(n) < 0.1] = -1
    K, V = rows(n, n, H), rows(n + 1, n, H)
    want = rng.integers(0, 256, (n_pages, H, page // 16, R.BLOCK)).astype(np.uint8)
    data = torch.from_numpy(want.copy()).cuda()
    R.store(want, page, slots, K, V)
    with B.Plan(1, 1) as p:
        p.qcache_append(bf(K), bf(V), i32(slots), data, page)
        assert p.status() == B.IKBO_OK
    assert R.nan_safe_equal(data.cpu().numpy(), want)


def test_append_of_strided_rows_and_of_none():
    H, n, page = 4, 33, 16
    wide = torch.randn(n, 3 * H * 128 + 8, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    K, V = (wide[:, a:a + H * 128].view(n, H, 128) for a in (H * 128, 2 * H * 128))
    slots = np.arange(n, dtype=np.int32)[::-1].copy()
    want = np.zeros((3, H, 1, R.BLOCK), np.uint8)
    data = torch.from_numpy(want.copy()).cuda()
    R.store(want, page, slots, K.float().cpu().numpy(), V.float().cpu().numpy())
    with B.Plan(1, 1) as p:
        p.qcache_append(K[:0], V[:0], i32([]), data, page)
        assert p.launches() == 0 and not data.any()
        p.qcache_append(K, V, i32(slots), data, page)
        assert R.nan_safe_equal(data.cpu().numpy(), want)
        one = torch.from_numpy(np.zeros_like(want)).cuda()
        p.qcache_append(K[4:5], V[4:5], i32(slots[4:5]), one, page)
        ref = np.zeros_like(want)
        R.store(ref, page, slots[4:5], K[4:5].float().cpu().numpy(), V[4:5].float().cpu().numpy())
        assert R.nan_safe_equal(one.cpu().numpy(), ref)
        for bad in (lambda: p.qcache_append(K, V.contiguous(), i32(slots), data, page),
                    lambda: p.qcache_append(K[:, ::2], V[:, ::2], i32(slots), data, page),
                    lambda: p.qcache_append(K, V, i32(slots[:-1]), data, page),
                    lambda: p.qcache_append(K, V, i32(slots), data, 32),
                    lambda: p.qcache_append(K.float(), V.float(), i32(slots), data, page)):
            with pytest.raises(ValueError):
                bad()


def test_append_leaves_out_slots_out_of_range():
    K, V = rows(1, 4, 2), rows(2, 4, 2)
    data = torch.full((2, 2, 1, R.BLOCK), 9, dtype=torch.uint8, device="cuda")
    want = data.cpu().numpy().copy()
    R.store(want, 16, [-1, 31, -1, -1], K, V)
    with B.Plan(1, 1) as p:
        p.qcache_append(bf(K), bf(V), i32([32, 31, -2, 2**31 - 1]), data, 16)
        assert p.status() == B.IKBO_ERR_CACHE
    assert R.nan_safe_equal(data.cpu().numpy(), want)


# ------------------------------------------------------------------ load
@pytest.mark.parametrize("lens,H,page", [([1], 1, 16), ([16, 17, 0, 15], 3, 16), ([200, 0, 1, 129], 2, 64),
                                         ([0, 0], 1, 32), ([5] * 300, 1, 16), ([2500], 2, 1024)])
def test_load_returns_the_values(lens, H, page):
    st = R.Store(len(lens), lens, H, page)
    data, table, ln = st.cuda()
    gap = np.arange(len(lens) + 1) * 3  # rows between the histories stay as they are
    off = np.concatenate([[0], np.cumsum(lens)]) + gap
    n = int(off[-1]) + 4
    K, V = (torch.full((n, H, 128), 11.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with B.Plan(1, 1) as p:
        p.qcache_load(data, page, table, ln, i32(off), K, V)
        assert p.status() == B.IKBO_OK
        V2 = torch.full_like(V, 11.0)
        p.qcache_load(data, page, table, ln, i32(off), None, V2)
    wk, wv = np.full((n, H, 128), 11.0, np.float32), np.full((n, H, 128), 11.0, np.float32)
    for u, (k, v) in enumerate(st.kv):
        wk[off[u]:off[u] + lens[u]], wv[off[u]:off[u] + lens[u]] = k, v
    assert np.array_equal(K.float().cpu().numpy(), wk)
    assert np.array_equal(V.float().cpu().numpy(), wv) and torch.equal(V, V2)


def test_load_cuts_and_reports():
    st = R.Store(1, [40, 20], 1, 16)
    data, table, ln = st.cuda()
    K, V = (torch.full((60, 1, 128), 11.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with B.Plan(1, 1) as p:
        p.qcache_load(data, 16, table, ln, i32([0, 33, 53]), K, V)  # the first has 33 rows only
        assert p.status() == B.IKBO_ERR_CACHE
        assert np.array_equal(K[:33].float().cpu().numpy(), st.kv[0][0][:33])
        assert np.array_equal(K[33:53].float().cpu().numpy(), st.kv[1][0])
        assert bool((K[53:] == 11.0).all())
        for off in ([0, 40, 61], [-1, 39, 59], [0, 70, 60]):
            K.fill_(11.0)
            p.qcache_load(data, 16, table, ln, i32(off), K, V)
            assert p.status() == B.IKBO_ERR_CACHE
        K.fill_(11.0)
        table[0, 1] = st.n_pages
        p.qcache_load(data, 16, table, ln, i32([0, 40, 60]), K, V)
        assert p.status() == B.IKBO_ERR_CACHE
        assert bool((K[16:32] == 11.0).all()) and np.array_equal(K[32:40].float().cpu().numpy(), st.kv[0][0][32:])
        ln[1] = -5
        p.qcache_load(data, 16, table, ln, i32([0, 40, 60]), K, V)
        assert p.status() == B.IKBO_ERR_CACHE
