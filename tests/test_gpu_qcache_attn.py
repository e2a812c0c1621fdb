"""Broadcast attention over the 4-bit cache against the definition in 64 bits
(qcache_util.attend derives the bound of every element)."""
import math

import numpy as np
import pytest
import torch

import qcache_util as R
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_qcache import Tables, bf, i32

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)

# The attention's three variants, reached by sizes alone: query rows a user
# (candidates times Lq) and the bound on the tokens, which may be any.
VARIANTS = {"registers": dict(c=1, Lq=8, Lkv=None), "tiles": dict(c=12, Lq=24, Lkv=8_000_000),
            "decoded": dict(c=9, Lq=128, Lkv=2000)}
each_variant = pytest.mark.parametrize("variant", list(VARIANTS))


def queries(seed, n, H, Lq, big=1.0):
    return R.bf16(np.random.default_rng(seed).standard_normal((n, H, Lq, 128)) * big)


def check(O, lse, Q, kv, m, H_kv, scale=SCALE):
    O64, l64, bound = R.attend(Q, kv, m, H_kv, scale)
    inside = np.array([0 <= int(u) < len(kv) for u in m])
    got = O.double().cpu().numpy()
    over = np.abs(got - O64) - bound
    assert np.all(over[inside] <= 0), float(np.nanmax(over[inside]))
    if lse is not None:
        g = lse.double().cpu().numpy()[inside]
        w = l64[inside]
        assert np.array_equal(np.isneginf(g), np.isneginf(w))
        fine = np.isfinite(w)
        # the scores' error (2^-16 of the largest |q||k|: at most 1e-2 here), log and the last rounding
        assert np.all(np.abs(g[fine] - w[fine]) <= 1e-4 * (1 + np.abs(w[fine])))


def attend(p, Q, st, lse=True, Lkv=None, scale=None, stream=None):
    data, table, ln = st.cuda()
    q = bf(Q)
    O = torch.full_like(q, float("nan"))
    L = torch.full(Q.shape[:3], float("nan"), device="cuda") if lse else None
    if stream is not None:
        torch.cuda.synchronize()
    p.attn_qcache_forward(q, data, st.page, table, ln, O, lse=L, Lkv=Lkv, scale=scale, stream=stream)
    return O, L


CASES = [
    # lens, cands per user, H, H_kv, Lq, page
    ([1], [1], 1, 1, 8, 16),
    ([15, 16, 17], [1, 1, 1], 2, 2, 8, 16),
    ([0, 33, 0], [2, 1, 0], 1, 1, 8, 16),
    ([1000], [1], 8, 8, 8, 64),
    ([700, 64, 0, 65, 1], [3, 0, 2, 1, 5], 2, 1, 16, 32),
    ([3000, 129], [1, 2], 8, 2, 24, 128),
    ([5000], [1], 4, 1, 8, 1024),
    ([40] * 70, [1] * 70, 2, 2, 8, 16),
    ([130, 0, 128], [2, 2, 2], 1, 1, 128, 16),
    ([300, 1, 257], [40, 1, 30], 2, 2, 16, 64),
    ([64, 500], [9, 8], 4, 2, 40, 32),
    ([1, 1, 2], [30, 40, 50], 3, 1, 8, 16),
    ([2500], [3], 4, 1, 16, 64),
    ([700, 0, 129, 1], [70, 2, 1, 80], 2, 2, 16, 32),
]


@pytest.mark.parametrize("bound", ["sum", "large"])
@pytest.mark.parametrize("lens,cands,H,H_kv,Lq,page", CASES)
def test_against_the_definition(lens, cands, H, H_kv, Lq, page, bound):
    """With the sum of the lengths as Lkv, and with a bound so large that every request of more
    than 16 rows a user goes through the tile kernel (up to 512)."""
    st = R.Store(sum(lens) + H, lens, H_kv, page)
    m = np.repeat(np.arange(len(lens)), cands)
    m = np.random.default_rng(1).permutation(m).astype(np.int32)
    Q = queries(2, len(m), H, Lq)
    Lkv = max(1, sum(lens)) if bound == "sum" else 1_000_000
    with B.Plan(len(m), len(lens), H) as p:
        p.plan(i32(m), len(lens), H, Lq)
        O, lse = attend(p, Q, st, Lkv=Lkv)
        assert p.status() == B.IKBO_OK
        check(O, lse, Q, st.kv, m, H_kv)
        O2, _ = attend(p, Q, st, lse=False, Lkv=Lkv)
        assert torch.equal(O, O2)  # bit for bit, with or without the log-sum-exp


@each_variant
def test_peaked_scores_and_other_scales(variant):
    """Scores of several hundred: the reference maximum moves; a scale of its own."""
    v = VARIANTS[variant]
    Lq, Lkv = v["Lq"], v["Lkv"]
    st = R.Store(8, [600, 100], 2, 16, outlier=8.0)
    m = np.repeat(np.arange(2), v["c"]).astype(np.int32)
    Q = queries(5, len(m), 2, Lq, big=4.0)
    with B.Plan(len(m), 2, 2) as p:
        p.plan(i32(m), 2, 2, Lq)
        for scale in (SCALE, 0.01, 0.5):
            O, _ = attend(p, Q, st, lse=False, Lkv=Lkv, scale=scale)
            check(O, None, Q, st.kv, m, 2, scale)


@each_variant
def test_candidates_without_a_user_keep_their_rows(variant):
    v = VARIANTS[variant]
    Lq = v["Lq"]
    st = R.Store(4, [50, 20], 1, 16)
    m = np.repeat([1, 7, 0, -1, 1, 0, 1, 1], v["c"]).astype(np.int32)
    if variant == "registers":
        m = m[:4]
    Q = queries(6, len(m), 1, Lq)
    with B.Plan(len(m), 2, 1) as p:
        p.plan(i32(m), 2, 1, Lq)
        O, lse = attend(p, Q, st, Lkv=v["Lkv"])
        assert p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE
        check(O, lse, Q, st.kv, m, 1)
        out = torch.from_numpy((m < 0) | (m > 1))
        assert bool(torch.isnan(O[out]).all()) and bool(torch.isnan(lse[out]).all())


@each_variant
def test_values_that_are_not_finite(variant):
    """A NaN in one user's values reaches that user's rows and no others; an
    infinite query makes its own row NaN."""
    Lq, c, Lkv = (VARIANTS[variant][k] for k in ("Lq", "c", "Lkv"))
    st = R.Store(7, [40, 40, 40], 1, 16)
    st.data[st.table[1, 2], 0, 0, 1280 + 1024:1280 + 1040] = 0xFF  # a value's pairs of user 1's token 32
    m = np.repeat(np.arange(3), c).astype(np.int32)
    Q = queries(6, 3 * c, 1, Lq)
    Q[2 * c, 0, 3, 5] = np.inf
    with B.Plan(3 * c, 3, 1) as p:
        p.plan(i32(m), 3, 1, Lq)
        O, _ = attend(p, Q, st, Lkv=Lkv)
    nan = torch.isnan(O).cpu().numpy()
    assert nan[c:2 * c].all() and not nan[:c].any()
    rows = nan[2 * c:].any(-1)
    assert rows[0, 0, 3] and rows.sum() == 1


@each_variant
def test_broken_tables_are_reported(variant):
    Lq, c, bound = (VARIANTS[variant][k] for k in ("Lq", "c", "Lkv"))
    m = np.repeat(np.arange(2), c).astype(np.int32)
    Q = queries(6, 2 * c, 1, Lq)

    def run(change, Lkv=bound):
        st = R.Store(9, [40, 300], 1, 16)
        kv = list(st.kv)
        change(st)
        with B.Plan(2 * c, 2, 1) as p:
            p.plan(i32(m), 2, 1, Lq)
            O, _ = attend(p, Q, st, Lkv=Lkv)
            assert p.status() == B.IKBO_ERR_CACHE
        return O, kv

    def page(st):
        st.table[1, 3] = st.n_pages

    def page_below(st):
        st.table[1, 0] = -1

    for change in (page, page_below):
        O, kv = run(change)
        check(O[:c], None, Q[:c], kv, m[:c], 1)  # the other user's rows

    def length(st):
        st.lens[1] = st.table.shape[1] * 16 + 1

    O, kv = run(length)
    check(O, None, Q, [kv[0], (kv[1][0][:0], kv[1][1][:0])], m, 1)
    if variant != "tiles":  # a bound below the sum (the tile kernel takes such short histories with a large one only)
        run(lambda st: None, Lkv=339)


def test_refusals_of_the_planned_request():
    st = R.Store(9, [20], 2, 16)
    data, table, ln = st.cuda()
    q = bf(queries(1, 2, 3, 8))
    with B.Plan(2, 1, 4) as p:
        with pytest.raises(B.IkboError) as e:
            p.attn_qcache_forward(q[:, :2].contiguous(), data, 16, table, ln, q[:, :2].contiguous())
        assert e.value.code == B.IKBO_ERR_NOT_PLANNED
        p.plan(i32([0, 0]), 1, 2, 8)
        with pytest.raises(ValueError):
            p.attn_qcache_forward(q, data, 16, table, ln, torch.empty_like(q))  # 3 heads
        ok = bf(queries(1, 2, 2, 8))
        with pytest.raises(ValueError):
            p.attn_qcache_forward(ok, data, 16, table, torch.cat([ln, ln]), torch.empty_like(ok))
        with pytest.raises(ValueError):
            p.attn_qcache_forward(ok, data, 32, table, ln, torch.empty_like(ok))
        with pytest.raises(ValueError):
            p.attn_qcache_forward(ok, data, 16, table, ln, torch.empty_like(ok), lse=torch.empty(2, 2, 7, device="cuda"))
        p.plan(i32([0, 0]), 1, 3, 8)
        L = B.load()
        assert L.ikbo_attn_qcache_forward(p.handle, q.data_ptr(), data.data_ptr(), st.n_pages, 16, 2, table.data_ptr(),
                                          table.shape[1], ln.data_ptr(), q.data_ptr(), None, 20, 128, 1.0, None) == \
            B.IKBO_ERR_INVALID_ARG  # 3 heads over 2


@each_variant
def test_other_stream_and_repeats(variant):
    v = VARIANTS[variant]
    Lq = v["Lq"]
    st = R.Store(11, [3000, 2000] if variant != "decoded" else [700, 300], 4, 64)
    m = np.repeat(np.arange(2), v["c"]).astype(np.int32)
    Q = queries(3, len(m), 4, Lq)
    with B.Plan(len(m), 2, 4) as p:
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        p.plan(i32(m), 2, 4, Lq, stream=s)
        outs = [attend(p, Q, st, Lkv=v["Lkv"], stream=s)[0] for _ in range(3)]
        assert p.status(s) == B.IKBO_OK
        check(outs[0], None, Q, st.kv, m, 4)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@each_variant
def test_graphs_keep_their_workspace(variant):
    """A captured call replays after a larger eager call has grown the plan's workspaces; a call
    that would have to allocate is refused under capture."""
    small, large = ([200, 90], [400, 3000])
    c, Lq = VARIANTS[variant]["c"], VARIANTS[variant]["Lq"]
    low, high = (290, 3400) if variant != "tiles" else (8_000_000, 8_000_000)
    m = np.repeat(np.arange(2), c).astype(np.int32)
    Q = queries(3, len(m), 2, Lq)
    a, b = R.Store(1, small, 2, 16), R.Store(2, large, 2, 64)
    with B.Plan(len(m), 2, 2) as p:
        p.plan(i32(m), 2, 2, Lq)
        data, table, ln = a.cuda()
        q, O = bf(Q), torch.zeros(Q.shape, dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(B.IkboError) as e:
                p.attn_qcache_forward(q, data, 16, table, ln, O, Lkv=low)
        assert e.value.code == B.IKBO_ERR_CUDA
        p.attn_qcache_forward(q, data, 16, table, ln, O, Lkv=low)
        first = O.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.attn_qcache_forward(q, data, 16, table, ln, O, Lkv=low)
        big, _ = attend(p, Q, b, Lkv=high)
        check(big, None, Q, b.kv, m, 2)
        O.zero_()
        graph.replay()
        assert torch.equal(O, first)
        check(O, None, Q, a.kv, m, 2)
        assert p.status() == B.IKBO_OK


def test_pages_behind_four_gigabytes():
    """Pages whose byte offsets need more than 32 bits, read by every variant and written."""
    page, H = 128, 8
    n_pages = 30000  # 4.9 GB
    assert B.ikbo_qcache_bytes(n_pages, page, H) > 2**32
    data = torch.full((n_pages, H, page // 16, R.BLOCK), 0xFF, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    K, V = R.bf16(rng.standard_normal((300, H, 128))), R.bf16(rng.standard_normal((300, H, 128)))
    table = np.array([[n_pages - 1, n_pages - 7, n_pages - 3]], np.int32)
    slots = table[0][np.arange(300) // page] * page + np.arange(300) % page
    values = [R.values(*R.quantise(x)) for x in (K, V)]
    with B.Plan(48, 1, H) as p:
        p.qcache_append(bf(K), bf(V), i32(slots), data, page)
        for n, Lq, Lkv in ((1, 8, 300), (24, 8, 1_000_000), (48, 24, 300)):
            m = np.zeros(n, np.int32)
            Q = queries(3, n, H, Lq)
            p.plan(i32(m), 1, H, Lq)
            q = bf(Q)
            O = torch.empty_like(q)
            p.attn_qcache_forward(q, data, page, i32(table), i32([300]), O, Lkv=Lkv)
            assert p.status() == B.IKBO_OK
            check(O, None, Q, [(values[0], values[1])], m, H)


def test_a_run_of_requests():
    """As a server uses them: lengths grow (and one history is dropped), keys are rotated at the
    positions the tables give, rows are stored, queries take their user's position, attention
    reads the cache; three requests over the same pages."""
    U, H, page, Lq = 3, 2, 16, 8
    rng = np.random.default_rng(21)
    freqs = B.ikbo_rope_frequencies(64, scaling="linear", factor=2.0)
    rope = B.Rope(64, freqs, interleaved=True)
    t = Tables(U, 12, page, 30, seed=4)
    data = torch.full((30, H, 1, R.BLOCK), 0xFF, dtype=torch.uint8, device="cuda")
    host = [(np.zeros((0, H, 128), np.float32), np.zeros((0, H, 128), np.float32)) for _ in range(U)]
    m = np.array([0, 2, 1, 0, 2, 0], np.int32)
    with B.Plan(6, U, H) as p:
        for new in ([40, 3, 100], [41, 0, 130], [90, 17, 131]):
            before = t.lens.copy()
            ok, slots, off, pos = t.resize(p, new, 160)
            assert ok
            n = int(off[-1])
            K, V = R.bf16(rng.standard_normal((n, H, 128))), R.bf16(rng.standard_normal((n, H, 128)))
            k, v = bf(K), bf(V)
            p.rope_forward(rope, k, k, start=pos[:n].contiguous())
            p.qcache_append(k, v, slots[:n].contiguous(), data, page)
            kr = k.float().cpu().numpy()
            ends = off.cpu().numpy()
            for u in range(U):
                a, b = ends[u], ends[u + 1]
                keep = min(int(before[u]), int(new[u]))
                host[u] = tuple(np.concatenate([x[:keep], R.values(*R.quantise(y[a:b]))])
                                for x, y in zip(host[u], (kr, V)))
                ref = R.rope_ref(K[a:b].astype(np.float64)[:, :, None, :], (int(before[u]) + np.arange(b - a))[:, None],
                                 freqs, True)[:, :, 0]
                assert np.all(np.abs(kr[a:b] - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5)
            p.plan(i32(m), U, H, Lq)
            q = bf(queries(new[0], 6, H, Lq))
            p.rope_forward(rope, q, q, start=t.dev[0], broadcast=True)
            O = torch.empty_like(q)
            p.attn_qcache_forward(q, data, page, t.dev[1], t.dev[0], O, Lkv=int(sum(new)) or 1)
            assert p.status() == B.IKBO_OK
            check(O, None, q.float().cpu().numpy(), host, m, H)
            # the same through the jagged entry point
            total = int(sum(new))
            Kj, Vj = (torch.zeros(total, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            offs = i32(np.concatenate([[0], np.cumsum(new)]))
            p.qcache_load(data, page, t.dev[1], t.dev[0], offs, Kj, Vj)
            Oj = torch.empty_like(q)
            p.attn_forward(q, Kj, Vj, offs, Oj)
            check(Oj, None, q.float().cpu().numpy(), host, m, H)


@pytest.mark.parametrize("variant,users,H,most", [
    ("registers", 33, 2, 90), ("registers", 150, 1, 90), ("registers", 700, 2, 60), ("registers", 2000, 1, 40),
    ("tiles", 33, 2, 90), ("tiles", 150, 1, 200), ("tiles", 700, 1, 60), ("tiles", 1300, 8, 20),
    ("decoded", 33, 1, 300), ("decoded", 400, 1, 40)])
def test_many_users(variant, users, H, most):
    """More users than a warp, a CTA's threads or a list in shared memory hold (1300 x 8 heads: over
    64 items for each CTA), one long history among short and empty ones, users without candidates."""
    c, Lq = {"registers": (1, 16), "tiles": (2, 24), "decoded": (9, 128)}[variant]
    rng = np.random.default_rng(users)
    lens = rng.integers(0, most, users)
    lens[[1, users - 1]] = 0, 1
    lens[users // 2] = 3000
    st = R.Store(users, lens.tolist(), H, 16)
    m = np.repeat(np.arange(users), c)
    m[rng.random(m.size) < 0.1] = users // 2  # some users without candidates, one with more
    m = rng.permutation(m).astype(np.int32)
    Q = np.tile(queries(4, 50, H, Lq), (-(-m.size // 50), 1, 1, 1))[:m.size]
    with B.Plan(m.size, users, H) as p:
        p.plan(i32(m), users, H, Lq)
        O, lse = attend(p, Q, st, Lkv=8_000_000 if variant == "tiles" else int(lens.sum()))
        assert p.status() == B.IKBO_OK
        O2, _ = attend(p, Q, st, lse=False, Lkv=8_000_000 if variant == "tiles" else int(lens.sum()))
        assert torch.equal(O, O2)
        assert not bool(torch.isnan(O).any())
        some = np.flatnonzero((m % max(1, users // 30) == 0) | (m == users - 1) | (m == 1))
        some = np.concatenate([some, np.flatnonzero(m == users // 2)[:5]])
        check(O[some], lse[some], Q[some], st.kv, m[some], H)


def test_a_loose_bound_costs_no_workspace():
    """Many rows a user, and the largest bound there is: no workspace of its size, the same rows."""
    st = R.Store(13, [300, 7], 2, 16)
    m = np.repeat(np.arange(2), 9).astype(np.int32)
    Q = queries(8, m.size, 2, 128)
    with B.Plan(m.size, 2, 2) as p:
        p.plan(i32(m), 2, 2, 128)
        before = torch.cuda.mem_get_info()[0]
        O, lse = attend(p, Q, st, Lkv=2**31 - 1)
        assert p.status() == B.IKBO_OK
        assert before - torch.cuda.mem_get_info()[0] < 2**30
        check(O, lse, Q, st.kv, m, 2)


@pytest.mark.parametrize("variant", ["registers", "tiles"])
def test_one_long_history(variant):
    """A history cut into a part for each of a hundred or more CTAs (registers: even parts)."""
    c, Lq = VARIANTS[variant]["c"], VARIANTS[variant]["Lq"]
    n = 40_000 if variant == "registers" else 60_000
    st = R.Store(17, [n], 1, 128)
    m = np.zeros(c, np.int32)
    Q = queries(9, c, 1, Lq, big=2.0)
    with B.Plan(c, 1, 1) as p:
        p.plan(i32(m), 1, 1, Lq)
        O, lse = attend(p, Q, st, Lkv=8_000_000)
        assert p.status() == B.IKBO_OK
        check(O, lse, Q, st.kv, m, 1)
        for _ in range(3):
            assert torch.equal(O, attend(p, Q, st, Lkv=8_000_000)[0])


def test_candidates_of_few_users():
    """Most users have none: the variant goes by the average, so a user's 2000 rows are many tiles of 16."""
    lens = [20] * 150 + [700] + [5] * 20
    st = R.Store(18, lens, 2, 16)
    m = np.concatenate([np.full(125, 150), np.arange(100, 140)]).astype(np.int32)
    m = np.random.default_rng(2).permutation(m)
    Q = queries(10, m.size, 2, 16)
    with B.Plan(m.size, len(lens), 2) as p:
        p.plan(i32(m), len(lens), 2, 16)
        O, lse = attend(p, Q, st, Lkv=sum(lens))
        assert p.status() == B.IKBO_OK
        check(O, lse, Q, st.kv, m, 2)
