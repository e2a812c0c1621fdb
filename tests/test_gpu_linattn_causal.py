"""An infinity or NaN in a row of linear attention reaches the rows that read it and no others: not earlier rows (in a
gradient of keys or values: later ones), whichever variant a call takes, nor other columns where it is a value's."""
import numpy as np
import pytest
import torch

import linattn_bounds as BD
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_linattn import SCALE, Data, bf, f32, plan, run_forward

pytestmark = pytest.mark.gpu

# rows of the first user, the row that is spoiled, and what the second user has
VARIANTS = {"row_by_row": ([8, 5], 3), "registers": ([90, 64], 50), "registers_second_chunk": ([90, 64], 80), "one_pass": ([60, 64], 21),
            "tiles": ([300, 130], 70), "tiles_second_chunk": ([300, 130], 181), "tiles_last_row": ([300, 130], 299), "cut": ([2600, 130], 1500)}
COLUMNS = [0, 3, 17, 64, 126, 127]


def spoil(x, t, h):
    x[t, h, COLUMNS[::2]] = np.nan
    x[t, h, COLUMNS[1::2]] = np.inf
    x[t, h, COLUMNS[3]] = -np.inf


@pytest.fixture(params=VARIANTS.values(), ids=VARIANTS.keys())
def case(request):
    lens, t = request.param
    return lens, t, Data(sum(lens), lens, 2, decay=[0.97, 0.5])


def run_backward(p, d, max_len):
    Q, K, V, decay, off = d.cuda()
    outs = [torch.empty_like(Q) for _ in range(3)]
    dS = torch.empty((len(d.off) - 1, d.H, 128, 128), device="cuda")
    p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off, max_len=max_len)
    return outs, dS


def rows_right(got, want, mass, rows, what):
    """The spoiled head's rows, and of the other head and the other user all."""
    for h, r in ((0, rows), (1, slice(None))):
        g = got.clone()[r, h]
        BD.near(g, want[r, h], mass[r, h], (what, h))


@pytest.mark.parametrize("operand", ["Q", "K", "V"])
def test_forward(case, operand):
    lens, t, d = case
    want, end, mass, emass = BD.forward(d, SCALE)
    spoil(getattr(d, operand), t, 0)
    others = [c for c in range(128) if c not in COLUMNS]
    apart = np.r_[0:t, lens[0]:sum(lens)] if operand != "Q" else np.r_[0:t, t + 1:sum(lens)]
    with plan() as p:
        O, S = run_forward(p, d, max_len=max(lens))
        rows_right(O, want, mass, apart, operand)
        if operand == "V":  # a value's columns are its own, then and in the state
            BD.near(O[..., others], want[..., others], mass[..., others], "other columns")
            assert not torch.isfinite(O[t:lens[0], 0][:, COLUMNS]).any() and not torch.isfinite(S[0, 0][:, COLUMNS]).any()
            BD.near_state(S[..., others], end[..., others], emass[..., others])
        elif operand == "K":
            assert not torch.isfinite(O[t:lens[0], 0]).any()
        BD.near_state(S[1], end[1], emass[1])
        BD.near_state(S[0, 1], end[0, 1], emass[0, 1])
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("operand", ["Q", "K", "V", "dO"])
def test_backward(case, operand):
    lens, t, d = case
    want, mass = BD.backward(d, SCALE)
    spoil(getattr(d, operand), t, 0)
    n = sum(lens)
    alone, none = np.r_[0:t, t + 1:n], np.r_[0:n]
    earlier, later = np.r_[0:t, lens[0]:n], np.r_[t + 1:n]
    apart = {"Q": (none, later, later), "K": (earlier, none, alone), "V": (earlier, alone, none), "dO": (alone, later, later)}[operand]
    with plan() as p:
        outs, dS = run_backward(p, d, max(lens))
        for k, name in enumerate(("dQ", "dK", "dV")):
            rows_right(outs[k], want[k], mass[k], apart[k], name)
        keep = dS if operand in "KV" else dS[1:]
        BD.near_state(keep, want[3][-len(keep):], mass[3][-len(keep):])
        assert p.status() == B.IKBO_OK


def test_what_overflows_by_itself_stays_where_it_is():
    """Outputs beyond bf16's range, without an infinity among the inputs."""
    d = Data(8, [300], 1, start=False, decay=[0.9])
    d.Q[40] *= 2.0 ** 100
    d.V[:, 0, 5] *= 2.0 ** 40
    want, _, mass, _ = BD.forward(d, SCALE)
    with plan() as p:
        O, _ = run_forward(p, d, max_len=300)
        big = np.abs(want) >= 2.0 ** 128
        assert big.any() and torch.isinf(O[torch.from_numpy(big).cuda()]).all()
        near = torch.where(torch.from_numpy(big).cuda(), 0, O)
        BD.near(near, np.where(big, 0, want), mass)
