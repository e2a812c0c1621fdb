"""Linear attention with a decay, its gradient, and the candidates' reads of the
states, against the definition row by row in 64 bits.

Tolerances.  Outputs in bf16 go through three roundings to bf16, each at most 2^-8 of
a term: the products q.k with their decay, the state as an operand, the output.  They
are independent, so in the 2-norm over a tensor they come to less than
sqrt(3) 2^-8 / sqrt(3) = 2^-8 (a rounding's mean square is a third of its largest);
2^-7 is asked for, and of each element 2^-8 |o| + 2^-7 of the sum of magnitudes that
makes it up.  States are held in fp32; a term is off by 2^-17 (the two bf16 parts of a
decayed value), the decay by 2^-22 a power, and each of at most 4000 rows' additions by
2^-24 of the partial sum: 2^-14 of the sum of magnitudes for an element, and 2^-16 in
the 2-norm (terms' signs are independent here).  With small whole numbers, decays of 0,
1/2 and 1, everything but the last rounding is exact, and results are compared bit by bit.
"""
import math

import numpy as np
import pytest
import torch

import linattn_util as R
from broadcast_gemm_attention_gb300 import binding as B
from qcache_util import bf16

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)


def plan():
    return B.Plan(4096, 512, 16)


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).cuda()


def f32(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def offsets_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def i32(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def host(t):
    return t.double().cpu().numpy()


def near(got, ref, what=""):
    """A bf16 tensor in the 2-norm."""
    got = host(got)
    assert np.all(np.isfinite(got)), what
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= 2.0 ** -7 * norm + 1e-30, (what, np.linalg.norm(got - ref) / norm)


def near_state(got, ref, mass, what=""):
    got = host(got)
    assert np.all(np.abs(got - ref) <= 2.0 ** -14 * mass + 1e-30), what
    assert np.linalg.norm(got - ref) <= 2.0 ** -16 * np.linalg.norm(ref) + 1e-30, what


class Data:
    def __init__(self, seed, lens, H, start=True, spare=0, whole=False, decay=None):
        rng = np.random.default_rng(seed)
        self.off = offsets_of(lens)
        n = int(self.off[-1]) + spare
        draw = (lambda s: rng.integers(-1, 2, s).astype(np.float32)) if whole else (lambda s: bf16(rng.standard_normal(s)))
        self.Q, self.K, self.V, self.dO = (draw((n, H, D)) for _ in range(4))
        shape = (len(lens), H, D, D)
        self.S = (rng.integers(-3, 4, shape) if whole else rng.standard_normal(shape) * 2).astype(np.float32) if start else None
        self.dS = (rng.integers(-3, 4, shape) if whole else rng.standard_normal(shape)).astype(np.float32) if start else None
        few = [1.0, 0.5, 0.0] if whole else [0.97, 1.0, 0.5, 0.0, 0.999]
        self.decay = np.array(decay if decay is not None else [few[h % len(few)] for h in range(H)], dtype=np.float32)
        self.H, self.n = H, n

    def cuda(self):
        return bf(self.Q), bf(self.K), bf(self.V), f32(self.decay), i32(self.off)


def run_forward(p, d, queries=True, scale=SCALE, max_len=0, keep=True, stream=None):
    Q, K, V, decay, off = d.cuda()
    O = torch.full_like(Q, -7.0) if queries else None
    last = torch.full((len(d.off) - 1, d.H, D, D), float("nan"), device="cuda") if keep else None
    p.linattn_forward(Q if queries else None, K, V, decay, O, state_in=f32(d.S), state_out=last, offsets=off, max_len=max_len, scale=scale,
                      stream=stream)
    return O, last


LENS = [[1], [0], [2, 0, 3], [5], [63], [64], [65], [0, 130, 1, 0, 64], [127, 129], [300, 7, 0, 0, 64, 200]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,start", [(1, False), (5, True)])
def test_forward(lens, H, start):
    d = Data(sum(lens) + H, lens, H, start, spare=3)
    ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, SCALE)
    mass = R.weights(d.K, d.V, d.decay, d.off, d.S)
    with plan() as p:
        for max_len in {0, max(max(lens), 1)}:
            O, S = run_forward(p, d, max_len=max_len)
            near(O[:d.off[-1]], ref[:d.off[-1]])
            near_state(S, last, mass)
            assert torch.all(O[d.off[-1]:] == -7.0)  # rows behind the last sequence
            _, S2 = run_forward(p, d, queries=False, max_len=max_len)
            near_state(S2, last, mass)
            O3, _ = run_forward(p, d, keep=False, max_len=max_len)
            assert torch.equal(O3, O)
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("lens", [[1], [4, 1, 0, 3], [64], [65], [40, 0, 129], [200], [1100, 3]], ids=str)
def test_whole_numbers_are_exact(lens):
    """Every product, sum and state is a whole number (or half of one, and so on) that fits its type."""
    d = Data(7, lens, 3, whole=True)
    # decay 1/2: powers of two below 1 times whole numbers; the products with queries stay exact in 24 bits
    # only near the diagonal, so that head is compared where the sums are short
    ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, 1.0)
    gq = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, d.S, d.dS, 1.0)
    exact = [0, 2] if max(lens) <= 128 else [2]  # |q.k| <= 128 and |S| <= 3 + rows: whole numbers of 8 bits up to 256
    with plan() as p:
        O, S = run_forward(p, d, scale=1.0, max_len=max(lens))
        Q, K, V, decay, off = d.cuda()
        dQ, dK, dV = (torch.full_like(Q, float("nan")) for _ in range(3))
        dS = torch.full_like(S, float("nan"))
        p.linattn_backward(Q, K, V, bf(d.dO), decay, dQ, dK, dV, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off,
                           scale=1.0)
        assert np.array_equal(host(S)[:, [0, 2]], last[:, [0, 2]])
        assert np.array_equal(host(dS)[:, [0, 2]], gq[3][:, [0, 2]])
        for got, want in ((O, ref), (dQ, gq[0]), (dK, gq[1]), (dV, gq[2])):
            assert np.array_equal(host(got)[:, exact], bf16(want[:, exact]).astype(np.float64))


@pytest.mark.parametrize("lens", [[1], [3, 0, 2], [64], [0, 65, 130], [190, 1]], ids=str)
@pytest.mark.parametrize("start", [False, True])
def test_backward(lens, start):
    d = Data(11 + sum(lens), lens, 4, start, spare=2)
    dQ64, dK64, dV64, dS64 = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, d.S, d.dS, SCALE)
    mass = R.backward(*(np.abs(x) for x in (d.Q, d.K, d.V, d.dO)), d.decay, d.off, None if d.S is None else np.abs(d.S),
                      None if d.dS is None else np.abs(d.dS), SCALE)[3]
    with plan() as p:
        Q, K, V, decay, off = d.cuda()
        outs = [torch.full_like(Q, -7.0) for _ in range(3)]
        dS = torch.full((len(lens), d.H, D, D), float("nan"), device="cuda")
        kw = dict(state_in=f32(d.S), d_state_out=f32(d.dS), offsets=off)
        p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, d_state_in=dS, **kw)
        end = d.off[-1]
        for got, want, name in zip(outs, (dQ64, dK64, dV64), ("dQ", "dK", "dV")):
            near(got[:end], want[:end], name)
            assert torch.all(got[end:] == -7.0)
        near_state(dS, dS64, mass)
        # any of them alone
        for k in range(4):
            alone = [torch.full_like(Q, -7.0) if k == j else None for j in range(3)]
            dS1 = torch.full_like(dS, float("nan")) if k == 3 else None
            p.linattn_backward(Q, K, V, bf(d.dO), decay, *alone, d_state_in=dS1, **kw)
            assert torch.equal(dS1 if k == 3 else alone[k], dS if k == 3 else outs[k])
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("lens,H", [([3, 0, 8, 1, 16, 17, 7, 9, 15], 2), ([64, 33, 48, 31], 3), ([300] + [1, 0, 5, 2] * 12, 1), ([2] * 90, 4)],
                         ids=["few", "blocks", "one_long", "many"])
def test_gradient_of_few_rows(lens, H):
    """In one pass: every set of gradients is the same, and that of the definition."""
    d = Data(50 + len(lens), lens, H, spare=3)
    g64 = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, d.S, d.dS, SCALE)
    mass = R.backward(*(np.abs(x) for x in (d.Q, d.K, d.V, d.dO)), d.decay, d.off, np.abs(d.S), np.abs(d.dS), SCALE)[3]
    with plan() as p:
        Q, K, V, decay, off = d.cuda()
        dO, s_in, ds_out = bf(d.dO), f32(d.S), f32(d.dS)
        full = None
        for want in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 1, 1, 0)):
            outs = [torch.full_like(Q, 5.0) if w else None for w in want[:3]] + [torch.full_like(s_in, float("nan")) if want[3] else None]
            before = p.launches()
            p.linattn_backward(Q, K, V, dO, decay, *outs[:3], state_in=s_in, d_state_out=ds_out, d_state_in=outs[3], offsets=off)
            assert p.launches() == before + 1
            if full is None:
                full = outs
                n = int(d.off[-1])
                for got, ref, name in zip(outs, g64, ("dQ", "dK", "dV")):
                    near(got[:n], ref[:n], name)
                    assert torch.all(got[n:] == 5.0)
                near_state(outs[3], g64[3], mass)
            for got, same in zip(outs, full):
                assert got is None or torch.equal(got, same)
        # without states
        outs, dS = [torch.empty_like(Q) for _ in range(3)], torch.full_like(s_in, float("nan"))
        p.linattn_backward(Q, K, V, dO, decay, *outs, d_state_in=dS, offsets=off)
        zero = np.zeros_like(d.S)
        ref = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, zero, zero, SCALE)
        for got, want, name in zip(outs, ref, ("dQ", "dK", "dV")):
            near(got[:n], want[:n], name)
        near_state(dS, ref[3], mass)
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("lens,H", [([2000], 1), ([900, 0, 2500], 2)], ids=str)
def test_histories_in_segments(lens, H):
    """Few long histories are cut; the start comes in and the end goes out in place."""
    d = Data(3, lens, H, decay=[0.995, 1.0][:H])
    ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, SCALE)
    mass = R.weights(d.K, d.V, d.decay, d.off, d.S)
    g64 = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, d.S, d.dS, SCALE)
    gmass = R.backward(*(np.abs(x) for x in (d.Q, d.K, d.V, d.dO)), d.decay, d.off, np.abs(d.S), np.abs(d.dS), SCALE)[3]
    with plan() as p:
        Q, K, V, decay, off = d.cuda()
        O, S = torch.empty_like(Q), f32(d.S)
        p.linattn_forward(Q, K, V, decay, O, state_in=S, state_out=S, offsets=off)
        assert p.launches() == 3  # the segments' parts, their joining, the outputs
        near(O, ref)
        near_state(S, last, mass)
        again, S2 = torch.empty_like(Q), f32(d.S)
        p.linattn_forward(Q, K, V, decay, again, state_in=S2, state_out=S2, offsets=off)
        assert torch.equal(again, O) and torch.equal(S2, S)
        S3 = f32(d.S)
        p.linattn_forward(None, K, V, decay, None, state_in=S3, state_out=S3, offsets=off)
        near_state(S3, last, mass)
        outs, dS = [torch.empty_like(Q) for _ in range(3)], torch.empty_like(S)
        p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off)
        for got, want, name in zip(outs, g64, ("dQ", "dK", "dV")):
            near(got, want, name)
        near_state(dS, g64[3], gmass)
        assert p.status() == B.IKBO_OK


def test_again_and_again():
    """The tile kernel's warps hand over to each other differently every time; results and status do not."""
    d = Data(17, [3000, 130, 700], 2, decay=[0.995, 0.9])
    with plan() as p:
        O, S = run_forward(p, d)
        Q, K, V, decay, off = d.cuda()
        dO, s_in, ds_out = bf(d.dO), f32(d.S), f32(d.dS)
        O2, S2, S3 = torch.empty_like(O), torch.empty_like(S), torch.empty_like(S)
        g = [torch.empty_like(Q) for _ in range(3)]
        p.linattn_backward(Q, K, V, dO, decay, *g, state_in=s_in, d_state_out=ds_out, d_state_in=S3, offsets=off)
        first = [t.clone() for t in (*g, S3)]
        _, alone = run_forward(p, d, queries=False)
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(300):
            p.linattn_forward(Q, K, V, decay, O2, state_in=s_in, state_out=S2, offsets=off)
            p.linattn_forward(None, K, V, decay, None, state_in=s_in, state_out=S3, offsets=off)
            wrong += (O2 != O).sum() + (S2 != S).sum() + (S3 != alone).sum()
            p.linattn_backward(Q, K, V, dO, decay, *g, state_in=s_in, d_state_out=ds_out, d_state_in=S3, offsets=off)
            for a, b in zip((*g, S3), first):
                wrong += (a != b).sum()
        assert p.status() == B.IKBO_OK and int(wrong) == 0


def test_inputs_that_change_right_before_and_after_a_call():
    """A cut history's launches may be set up while the one before ends: not before what is ahead of the call, nor past what is behind it."""
    lens = [4000, 900]
    both = [Data(seed, lens, 2, decay=[0.995, 0.9]) for seed in (31, 32)]
    with plan() as p:
        want = [run_forward(p, d) for d in both]
        ins = [(*d.cuda()[:3], f32(d.S)) for d in both]
        decay, off = both[0].cuda()[3:]
        Q, K, V, S = (torch.zeros_like(t) for t in ins[0])
        O = torch.zeros_like(Q)
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")

        def once(i):
            for to, x in zip((Q, K, V, S), ins[i]):
                to.copy_(x)
            before = p.launches()
            p.linattn_forward(Q, K, V, decay, O, state_in=S, state_out=S, offsets=off)  # (the state in its place)
            assert p.launches() == before + 3
            for to in (Q, K, V):
                to.fill_(7.0)
            wrong.add_((O != want[i][0]).sum() + (S != want[i][1]).sum())
            O.zero_()

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


def test_events_one_by_one_are_the_whole():
    """A history taken in at once, in pieces, and token by token ends in the same state."""
    d = Data(5, [150], 3)
    with plan() as p:
        Q, K, V, decay, _ = d.cuda()
        O, S = run_forward(p, d)
        one, many = f32(d.S), f32(d.S)
        O1, O2 = torch.empty_like(Q), torch.empty_like(Q)
        for r in range(150):
            p.linattn_forward(Q[r:r + 1], K[r:r + 1], V[r:r + 1], decay, O1[r:r + 1], state_in=one, state_out=one)
        for a, b in ((0, 40), (40, 104), (104, 150)):
            p.linattn_forward(Q[a:b], K[a:b], V[a:b], decay, O2[a:b], state_in=many, state_out=many)
        ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, SCALE)
        mass = R.weights(d.K, d.V, d.decay, d.off, d.S)
        for o, s in ((O, S), (O1, one), (O2, many)):
            near(o, ref)
            near_state(s, last, mass)


def test_slices_of_a_projection_and_dense_rows():
    U, L, H = 3, 70, 2
    rng = np.random.default_rng(0)
    qkv = bf(rng.standard_normal((U * L, 3, H, D)))
    Q, K, V = qkv[:, 0], qkv[:, 1], qkv[:, 2]
    decay = f32([0.9, 1.0])
    wide = torch.zeros((U * L, 2, H, D), dtype=torch.bfloat16, device="cuda")
    with plan() as p:
        p.linattn_forward(Q, K, V, decay, wide[:, 1], n_users=U)
        plain = torch.empty((U * L, H, D), dtype=torch.bfloat16, device="cuda")
        p.linattn_forward(Q.contiguous(), K.contiguous(), V.contiguous(), decay, plain, offsets=i32(offsets_of([L] * U)), max_len=L)  # (the variant goes by it)
        assert torch.equal(wide[:, 1], plain) and not wide[:, 0].any()
        g, dq = torch.zeros_like(qkv), bf(rng.standard_normal((U * L, H, D)))
        p.linattn_backward(Q, K, V, dq, decay, g[:, 0], g[:, 1], g[:, 2], n_users=U)
        outs = [torch.empty_like(plain) for _ in range(3)]
        p.linattn_backward(Q.contiguous(), K.contiguous(), V.contiguous(), dq, decay, *outs, n_users=U)
        for k in range(3):
            assert torch.equal(g[:, k], outs[k])
        with pytest.raises(B.IkboError):
            p.linattn_forward(Q, K, V, decay, plain, n_users=4)  # 210 rows are not four times as many


def test_no_rows_at_all():
    """Empty tensors: the states pass through, and nothing is asked of the rows' addresses."""
    S = torch.randn((3, 2, D, D), device="cuda")
    none = torch.empty((0, 2, D), dtype=torch.bfloat16, device="cuda")
    decay = f32([0.9, 1.0])
    with plan() as p:
        for off in (i32([0, 0, 0, 0]), None):
            out = torch.full_like(S, float("nan"))
            p.linattn_forward(none, none, none, decay, none, state_in=S, state_out=out, offsets=off)
            assert torch.equal(out, S)
            out.fill_(float("nan"))
            p.linattn_forward(None, none, none, decay, None, state_out=out, offsets=off, n_users=3)
            assert not out.any()
            out.fill_(float("nan"))
            p.linattn_backward(none, none, none, none, decay, none, none, none, state_in=S, d_state_out=S, d_state_in=out, offsets=off)
            near_state(out, host(S), np.abs(host(S)))
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("max_len", [0, 300])
def test_another_user_s_infinities_stay_there(max_len):
    """Rows beside a user's own, behind its last in the same tile, hold infinities and NaN."""
    lens = [100, 40, 131, 60]
    d = Data(19, lens, 2, spare=40)
    own = np.r_[0:100, 140:271]                  # the first and the third user's rows
    ref = {}
    with plan() as p:
        for bad in (False, True):
            if bad:
                for x in (d.Q, d.K, d.V, d.dO):
                    x[100:140:3] = np.inf
                    x[101:140:3] = np.nan
                    x[271:] = np.nan
            O, S = run_forward(p, d, max_len=max_len)
            Q, K, V, decay, off = d.cuda()
            outs, dS = [torch.empty_like(Q) for _ in range(3)], torch.empty_like(S)
            p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off,
                               max_len=max_len)
            got = [t[own].clone() for t in (O, *outs)] + [S[[0, 2]], dS[[0, 2]]]
            if bad:
                assert all(torch.equal(a, b) for a, b in zip(ref["is"], got))
            ref["is"] = got


def test_bad_offsets_are_reported_and_skipped():
    d = Data(9, [10, 10, 10], 2)
    ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, SCALE)
    mass = R.weights(d.K, d.V, d.decay, d.off, d.S)
    Q, K, V, decay, _ = d.cuda()
    with plan() as p:
        for bad in ([0, 10, 5, 30], [0, 10, 31, 30], [0, 10, -1, 30]):
            O, S = torch.full_like(Q, -7.0), torch.full((3, 2, D, D), float("nan"), device="cuda")
            p.linattn_forward(Q, K, V, decay, O, state_in=f32(d.S), state_out=S, offsets=i32(bad), max_len=25)
            assert p.status() == B.IKBO_ERR_CACHE and p.status() == B.IKBO_OK
            own = 5 if bad[2] == 5 else 10  # (there the third user's rows 5 .. 29 are sound by themselves, and two users write 5 .. 9)
            near(O[:own], ref[:own])
            near_state(S[:1], last[:1], mass[:1])
            assert np.array_equal(host(S[1]), d.S[1].astype(np.float64))  # taken for one without rows
        O, S = run_forward(p, d, max_len=9)  # longer than they were said to be
        assert p.status() == B.IKBO_ERR_CACHE
        assert torch.all(O == -7.0) and np.array_equal(host(S), d.S.astype(np.float64))


def test_captured_and_on_another_stream():
    d = Data(13, [1200], 2, decay=[0.99, 0.9])
    with plan() as p:
        O, S = run_forward(p, d)
        Q, K, V, decay, off = d.cuda()
        s_in = f32(d.S)
        O2, S2 = torch.zeros_like(Q), torch.zeros_like(S)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.linattn_forward(Q, K, V, decay, O2, state_in=s_in, state_out=S2, offsets=off)
        # a larger eager call moves the plan's workspace; the graph keeps its own
        big = Data(14, [6000], 4)
        run_forward(p, big)
        for _ in range(2):
            O2.zero_()
            S2.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(O2, O) and torch.equal(S2, S)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            O3, S3 = run_forward(p, d, stream=side)
        side.synchronize()
        assert torch.equal(O3, O) and torch.equal(S3, S)
        assert p.status() == B.IKBO_OK
    with plan() as p:  # a capture that would have to allocate is refused
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(B.IkboError):
                p.linattn_forward(Q, K, V, decay, O2, state_in=s_in, state_out=S2, offsets=off)


def test_a_wait_that_runs_out_is_reported_and_passes():
    """Every fourth CTA of the tile kernels waits for what never comes: the calls end, say so, and leave nothing behind."""
    d = Data(18, [700, 150, 30], 3, decay=[0.99, 0.9, 1.0])
    rng = np.random.default_rng(18)
    m = np.sort(rng.integers(0, 3, 200)).astype(np.int32)
    X, dO = bf16(rng.standard_normal((200, 3, 16, D))), bf16(rng.standard_normal((200, 3, 16, D)))
    with plan() as p:
        mm = i32(m)
        p.plan(mm, 3, 3, 16)
        O, S = run_forward(p, d)
        dX, dS, dS2 = torch.empty_like(bf(X)), torch.empty_like(S), torch.empty_like(S)
        p.linattn_read_backward(bf(X), S, bf(dO), dX, dS)
        assert p.status() == B.IKBO_OK
        for _ in range(3):
            B.ikbo_plan_set_timeout_ns(p.handle, 20_000_000)
            B.ikbo_plan_set_debug(p.handle, B.DEBUG_WITHHOLD_STATES)
            run_forward(p, d)
            assert p.status() == B.IKBO_ERR_TIMEOUT
            run_forward(p, d, queries=False)
            assert p.status() == B.IKBO_ERR_TIMEOUT
            p.linattn_read_backward(bf(X), S, bf(dO), dX, dS2)
            assert p.status() == B.IKBO_ERR_TIMEOUT
            B.ikbo_plan_set_timeout_ns(p.handle, 2_000_000_000)
            B.ikbo_plan_set_debug(p.handle, 0)
            O2, S2 = run_forward(p, d)
            p.linattn_read_backward(bf(X), S, bf(dO), dX, dS2)
            assert p.status() == B.IKBO_OK
            assert torch.equal(O2, O) and torch.equal(S2, S) and torch.equal(dS2, dS)


def test_many_users_of_a_few_rows():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, 400)
    lens[7] = 9
    d = Data(15, lens, 1)
    ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, SCALE)
    with plan() as p:
        O, S = run_forward(p, d, max_len=9)
        near(O, ref)
        near_state(S, last, R.weights(d.K, d.V, d.decay, d.off, d.S))


def test_more_histories_than_sms():
    """Each CTA of the tile kernel goes through several, most ending in a part of a chunk."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 400, 90)
    lens[[3, 40]] = 0, 256
    d = Data(16, lens, 4, decay=[0.99, 1.0, 0.7, 0.0])
    ref, last = R.forward(d.Q, d.K, d.V, d.decay, d.off, d.S, SCALE)
    g64 = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, d.S, d.dS, SCALE)
    gmass = R.backward(*(np.abs(x) for x in (d.Q, d.K, d.V, d.dO)), d.decay, d.off, np.abs(d.S), np.abs(d.dS), SCALE)[3]
    with plan() as p:
        O, S = run_forward(p, d, max_len=400)
        near(O, ref)
        near_state(S, last, R.weights(d.K, d.V, d.decay, d.off, d.S))
        _, S2 = run_forward(p, d, queries=False, max_len=400)
        near_state(S2, last, R.weights(d.K, d.V, d.decay, d.off, d.S))
        Q, K, V, decay, off = d.cuda()
        outs, dS = [torch.empty_like(Q) for _ in range(3)], torch.empty_like(S)
        p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off,
                           max_len=400)
        for got, want, name in zip(outs, g64, ("dQ", "dK", "dV")):
            near(got, want, name)
        near_state(dS, g64[3], gmass)
        assert p.status() == B.IKBO_OK


# ------------------------------------------------------------------- reads
def read_ref(X, S, m, scale, turned=False):
    out = np.zeros(X.shape)
    for i, u in enumerate(m):
        if 0 <= u < len(S):
            out[i] = scale * np.einsum("hld,hed->hle" if turned else "hld,hde->hle", X[i].astype(np.float64), S[u].astype(np.float64))
    return out


@pytest.mark.parametrize("n,U,H,Lq", [(1, 1, 1, 8), (5, 3, 2, 8), (40, 4, 3, 24), (70, 1, 2, 32), (9, 12, 1, 128), (300, 17, 4, 16),
                                      (700, 3, 8, 8)])
def test_reads(n, U, H, Lq):
    rng = np.random.default_rng(n)
    m = rng.integers(0, U, n).astype(np.int32)
    X, dO = bf16(rng.standard_normal((n, H, Lq, D))), bf16(rng.standard_normal((n, H, Lq, D)))
    S = (rng.standard_normal((U, H, D, D)) * 3).astype(np.float32)
    dS64, mass = np.zeros(S.shape), np.zeros(S.shape)
    for i, u in enumerate(m):
        dS64[u] += SCALE * np.einsum("hld,hle->hde", X[i].astype(np.float64), dO[i].astype(np.float64))
        mass[u] += SCALE * np.einsum("hld,hle->hde", np.abs(X[i]).astype(np.float64), np.abs(dO[i]).astype(np.float64))
    with plan() as p:
        mm = i32(m)
        p.plan(mm, U, H, Lq)
        x, s, do = bf(X), f32(S), bf(dO)
        O, dQ, dS = torch.full_like(x, float("nan")), torch.full_like(x, float("nan")), torch.full_like(s, float("nan"))
        p.linattn_read_forward(x, s, O)
        p.linattn_read_backward(x, s, do, dQ, dS)
        near(O, read_ref(X, S, m, SCALE))
        near(dQ, read_ref(dO, S, m, SCALE, turned=True))
        # exact products, fp32 sums
        assert np.all(np.abs(host(dS) - dS64) <= 2.0 ** -18 * mass)
        dS2 = torch.full_like(s, float("nan"))
        p.linattn_read_backward(x, None, do, None, dS2)
        assert torch.equal(dS, dS2)
        p.linattn_read_forward(x, s, x)  # in place
        assert torch.equal(x, O)
        assert p.status() == B.IKBO_OK


def test_reads_of_whole_numbers_are_exact():
    rng = np.random.default_rng(0)
    n, U, H, Lq = 33, 5, 2, 40
    m = np.sort(rng.integers(0, U - 1, n)).astype(np.int32)  # the last user has no candidates
    X, dO = (rng.integers(-2, 3, (n, H, Lq, D)).astype(np.float32) for _ in range(2))
    S = rng.integers(-100, 101, (U, H, D, D)).astype(np.float32)
    with plan() as p:
        mm = i32(m)
        p.plan(mm, U, H, Lq)
        O, dQ, dS = bf(X), bf(X), torch.full((U, H, D, D), float("nan"), device="cuda")
        p.linattn_read_forward(bf(X), f32(S), O, scale=0.5)
        p.linattn_read_backward(bf(X), f32(S), bf(dO), dQ, dS, scale=0.5)
        assert np.array_equal(host(O), bf16(read_ref(X, S, m, 0.5)).astype(np.float64))
        assert np.array_equal(host(dQ), bf16(read_ref(dO, S, m, 0.5, turned=True)).astype(np.float64))
        want = np.zeros(S.shape)
        for i, u in enumerate(m):
            want[u] += 0.5 * np.einsum("hld,hle->hde", X[i], dO[i])
        assert np.array_equal(host(dS), want)
        assert not dS[U - 1].any()


@pytest.mark.parametrize("counts,H,Lq", [
    ([1000] + [1] * 40, 2, 16),            # one user's run over most CTAs, then runs of one
    ([0, 3] * 30 + [300, 0, 0, 90], 3, 8),  # users without candidates between
    ([1] * 152, 1, 128), ([1] * 76, 2, 64), ([2] * 151, 1, 128), ([151], 1, 128), ([9, 143], 1, 128),  # a unit or two for each SM
    ([k % 4 for k in range(700)], 1, 32), ([1] * 1400, 2, 8), ([0] * 1300 + [5, 200], 3, 24)], ids=lambda x: f"{len(x)}u" if isinstance(x, list) else str(x))
def test_shares_of_uneven_users_are_exact(counts, H, Lq):
    """Runs of units shared between CTAs, in every way; twice, as counts go back to zero."""
    g = torch.Generator().manual_seed(len(counts))
    n, U = sum(counts), len(counts)
    m = torch.repeat_interleave(torch.arange(U), torch.tensor(counts))[torch.randperm(n, generator=g)].int().cuda()
    X, dO = (torch.randint(-2, 3, (n, H, Lq, D), generator=g).float().cuda() for _ in range(2))
    S = torch.randint(-9, 10, (U, H, D, D), generator=g).float().cuda()
    want = torch.zeros(S.shape, dtype=torch.float64, device="cuda")
    O64, dX64 = torch.empty(X.shape, dtype=torch.float64, device="cuda"), torch.empty(X.shape, dtype=torch.float64, device="cuda")
    for i in range(0, n, 64):
        x, do, u = X[i:i + 64].double(), dO[i:i + 64].double(), m[i:i + 64].long()
        want.index_add_(0, u, 0.5 * x.transpose(2, 3) @ do)
        O64[i:i + 64], dX64[i:i + 64] = 0.5 * x @ S[u].double(), 0.5 * do @ S[u].double().transpose(2, 3)
    with B.Plan(2048, 2048, 4) as p:
        p.plan(m, U, H, Lq)
        for _ in range(2):
            O, dX, dS = torch.full_like(X, 9.0).bfloat16(), torch.full_like(X, 9.0).bfloat16(), torch.full_like(S, float("nan"))
            p.linattn_read_forward(X.bfloat16(), S, O, scale=0.5)
            p.linattn_read_backward(X.bfloat16(), S, dO.bfloat16(), dX, dS, scale=0.5)
            assert torch.equal(dS.double(), want)
            assert torch.equal(O, O64.bfloat16()) and torch.equal(dX, dX64.bfloat16())
        assert p.status() == B.IKBO_OK


def test_a_candidate_out_of_range_keeps_its_rows():
    rng = np.random.default_rng(2)
    m = np.array([0, 7, 1, -1, 1], np.int32)
    X, S = bf16(rng.standard_normal((5, 2, 8, D))), rng.standard_normal((2, 2, D, D)).astype(np.float32)
    with plan() as p:
        mm = i32(m)
        p.plan(mm, 2, 2, 8)
        assert p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE
        O = torch.full((5, 2, 8, D), -7.0, dtype=torch.bfloat16, device="cuda")
        p.linattn_read_forward(bf(X), f32(S), O)
        inside = [0, 2, 4]
        near(O[inside], read_ref(X, S, m, SCALE)[inside])
        assert torch.all(O[[1, 3]] == -7.0)
        with pytest.raises(ValueError):
            p.linattn_read_forward(bf(X), f32(S[:1]), O)
    with plan() as p, pytest.raises(B.IkboError):
        p.linattn_read_forward(bf(X), f32(S), O)  # not planned


def test_a_request_with_its_gradients():
    """Histories into states, candidates read them, and the gradients all the way back."""
    rng = np.random.default_rng(4)
    U, H, Lq, lens = 3, 2, 8, [90, 0, 40]
    d = Data(21, lens, H, start=False, decay=[0.9, 0.99])
    m = np.array([0, 2, 0, 1, 2, 2], np.int32)
    X, dO = bf16(rng.standard_normal((6, H, Lq, D))), bf16(rng.standard_normal((6, H, Lq, D)))
    O64, S64 = R.forward(d.Q, d.K, d.V, d.decay, d.off, None, SCALE)
    dS64 = np.zeros(S64.shape)
    for i, u in enumerate(m):
        dS64[u] += SCALE * np.einsum("hld,hle->hde", X[i].astype(np.float64), dO[i].astype(np.float64))
    g64 = R.backward(d.Q, d.K, d.V, d.dO, d.decay, d.off, None, dS64, SCALE)
    with plan() as p:
        mm = i32(m)
        p.plan(mm, U, H, Lq)
        Q, K, V, decay, off = d.cuda()
        O, S = torch.empty_like(Q), torch.empty((U, H, D, D), device="cuda")
        p.linattn_forward(Q, K, V, decay, O, state_out=S, offsets=off)
        Y = torch.empty_like(bf(X))
        p.linattn_read_forward(bf(X), S, Y)
        near(Y, read_ref(X, S64, m, SCALE))
        dX, dS = torch.empty_like(Y), torch.empty_like(S)
        p.linattn_read_backward(bf(X), S, bf(dO), dX, dS)
        near(dX, read_ref(dO, S64, m, SCALE, turned=True))
        outs = [torch.empty_like(Q) for _ in range(3)]
        p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, d_state_out=dS, offsets=off)
        for got, want in zip(outs, g64):
            near(got, want)
        assert p.status() == B.IKBO_OK
