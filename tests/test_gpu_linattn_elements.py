"""Linear attention element by element: every output within the bound that linattn_bounds derives, each user's rows
128 at a time in the 2-norm, and whole numbers bit by bit, in every variant and where histories are cut for many users."""
import numpy as np
import pytest
import torch

import linattn_bounds as BD
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_linattn import SCALE, Data, bf, f32, plan, run_forward

pytestmark = pytest.mark.gpu


def run_backward(p, d, scale, max_len):
    Q, K, V, decay, off = d.cuda()
    outs = [torch.full_like(Q, float("nan")) for _ in range(3)]
    dS = torch.full((len(d.off) - 1, d.H, 128, 128), float("nan"), device="cuda")
    p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off, scale=scale,
                       max_len=max_len)
    return (*outs, dS)


def skewed(users, long, seed):
    """Users of 0 to 10 rows, and some long ones."""
    lens = np.random.default_rng(seed).integers(0, 11, users)
    lens[[1, -1]] = 0
    for u, n in long.items():
        lens[u] = n
    return [int(n) for n in lens]


VARIANTS = [([5, 8, 0, 3], 8, 1), ([64, 20, 0, 65, 95], 95, 1), ([40, 64, 1, 33, 16, 17], 64, 1), ([130, 0, 300, 128, 1, 400], 400, 1),
            ([500] * 60 + [120, 0] * 20, 500, 1), ([2500, 300], 2500, 3)]


@pytest.mark.parametrize("lens,max_len,launches", VARIANTS, ids=["row_by_row", "registers", "one_pass", "tiles", "many_tiles", "cut"])
def test_every_element(lens, max_len, launches):
    H = 5 if len(lens) < 50 else 3
    d = Data(70 + len(lens), lens, H, decay=[0.97, 1.0, 0.5, 0.0, 0.999][:H])
    t = [torch.from_numpy(x).cuda() for x in (d.Q, d.K, d.V, d.dO, d.decay)]
    S, dS = f32(d.S), f32(d.dS)
    a = [x.abs() for x in (*t[:4], S, dS)]
    with plan() as p:
        before = p.launches()
        O, last = run_forward(p, d, max_len=max_len)
        assert p.launches() == before + launches
        want, end, _ = BD.long_forward(*t[:3], t[4], d.off, S, SCALE)
        mass, emass, _ = BD.long_forward(*a[:3], t[4], d.off, a[4], SCALE)
        BD.near_long(O, want, mass)
        BD.near_blocks(O, want, d.off)
        assert torch.all((last.double() - end).abs() <= 2.0 ** -14 * emass)
        _, alone = run_forward(p, d, queries=False, max_len=max_len)
        assert torch.all((alone.double() - end).abs() <= 2.0 ** -14 * emass)
        got = run_backward(p, d, SCALE, max_len)
        want = BD.long_backward(*t[:4], t[4], d.off, S, dS, SCALE)
        mass = BD.long_backward(*a[:4], t[4], d.off, *a[4:], SCALE)
        for k, name in enumerate(("dQ", "dK", "dV")):
            BD.near_long(got[k], want[k], mass[k], name)
            BD.near_blocks(got[k], want[k], d.off, name)
        assert torch.all((got[3].double() - want[3]).abs() <= 2.0 ** -14 * mass[3])
        assert p.status() == B.IKBO_OK


# users past a warp's lanes whose segments are looked up, with and without two scans for an SM
CUT = [(70, 1, {0: 3000, 40: 2871}), (70, 3, {40: 6500, 66: 200}), (250, 1, {33: 5000, 64: 300}), (33, 2, {32: 7000})]


@pytest.mark.parametrize("users,H,long", CUT, ids=lambda x: str(x) if isinstance(x, int) else "+".join(map(str, x.values())))
def test_whole_numbers_of_many_users_cut(users, H, long):
    """Where few users' histories are far longer than the others', they alone are cut; in place, and every gradient, bit by bit."""
    d = whole(skewed(users, long, users), H, [1.0] * H)
    check_whole(d, max(long.values()), 3)


def test_whole_numbers_of_more_scans_than_sms():
    """Several scans a CTA, of up to two chunks: |S| <= 3 + 250 is held exactly as bf16, and so is |q.k| <= 128."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(60, 251, 70)]
    lens[3], lens[50], lens[69] = 0, 128, 250
    check_whole(whole(lens, 4, [1.0, 0.0, 1.0, 1.0]), 250, 1)


def whole(lens, H, decay):
    """Rows of -1, 0 (seven of ten) and 1."""
    d = Data(9, lens, H, whole=True, decay=decay)
    rng = np.random.default_rng(10)
    for x in (d.Q, d.K, d.V, d.dO):
        x *= rng.random(x.shape) < 0.45
    return d


def check_whole(d, max_len, launches):
    t = [torch.from_numpy(x).cuda() for x in (d.Q, d.K, d.V, d.dO, d.decay)]
    S, dS = f32(d.S), f32(d.dS)
    O64, end, seen = BD.long_forward(*t[:3], t[4], d.off, S, 1.0)
    g64 = BD.long_backward(*t[:4], t[4], d.off, S, dS, 1.0)
    assert max(seen, g64[4]) <= 256  # whole numbers of 8 bits, at every chunk's border
    with plan() as p:
        Q, K, V, decay, off = d.cuda()
        for queries in (True, False):
            state, O = f32(d.S), torch.full_like(Q, float("nan"))
            before = p.launches()
            p.linattn_forward(Q if queries else None, K, V, decay, O if queries else None, state_in=state, state_out=state, offsets=off,
                              max_len=max_len, scale=1.0)
            if queries:
                assert p.launches() == before + launches
                assert torch.equal(O, O64.to(torch.bfloat16))
            assert torch.equal(state.double(), end)
        before = p.launches()
        got = run_backward(p, d, 1.0, max_len)
        assert p.launches() == before + launches
        for k in range(3):
            assert torch.equal(got[k], g64[k].to(torch.bfloat16)), k
        assert torch.equal(got[3].double(), g64[3])
        assert p.status() == B.IKBO_OK
