"""The gradient of long histories, whatever the scale: what the states' gradients hold does not depend on it."""
import numpy as np
import pytest
import torch

import linattn_bounds as BD
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_linattn import Data, bf, f32, plan

pytestmark = pytest.mark.gpu


def gradients(p, d, scale, max_len):
    Q, K, V, decay, off = d.cuda()
    outs = [torch.full_like(Q, -7.0) for _ in range(3)]
    dS = torch.full((len(d.off) - 1, d.H, 128, 128), float("nan"), device="cuda")
    p.linattn_backward(Q, K, V, bf(d.dO), decay, *outs, state_in=f32(d.S), d_state_out=f32(d.dS), d_state_in=dS, offsets=off, scale=scale,
                       max_len=max_len)
    return outs, dS


@pytest.mark.parametrize("lens", [[200, 0, 130, 0], [0, 3000, 0]], ids=["whole", "cut"])
def test_a_user_without_rows_passes_its_gradient_on(lens):
    """d_state_in is d_state_out, bit by bit, beside users that have rows."""
    d = Data(40, lens, 3, decay=[0.9, 1.0, 0.3])
    with plan() as p:
        before = p.launches()
        _, dS = gradients(p, d, 0.3, max(lens))
        assert p.launches() == before + (3 if lens[1] else 1)
        none = [u for u, n in enumerate(lens) if n == 0]
        assert np.array_equal(dS[none].cpu().numpy(), d.dS[none])
        assert p.status() == B.IKBO_OK


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 1e-3, 2.0 ** 40])
@pytest.mark.parametrize("size", ["like the rows'", "far larger"])
@pytest.mark.parametrize("lens", [[150, 0, 300], [3000]], ids=["whole", "cut"])
def test_any_scale(lens, size, scale):
    """d_state_out as large as what the rows add to it, and so large that divided by a small scale it passes 2^128."""
    d = Data(41, lens, 1, decay=[0.998])
    d.dS = (d.dS.astype(np.float64) * scale * (2.0 ** (131 if scale < 1e-9 else 40) if size == "far larger" else 1.0)).astype(np.float32)
    want, mass = BD.backward(d, scale)
    with plan() as p:
        outs, dS = gradients(p, d, scale, max(lens))
        for got, w, m, name in zip(outs, want, mass, ("dQ", "dK", "dV")):
            BD.near(got, w, m, name)
        BD.near_state(dS, want[3], mass[3])
        assert p.status() == B.IKBO_OK


def test_no_user_has_rows():
    """In tiles too: states pass through, rows of no user are left alone."""
    d = Data(42, [0, 0, 0], 3, spare=200)
    Q, K, V, decay, off = d.cuda()
    with plan() as p:
        for queries in (True, False):
            O, S = torch.full_like(Q, -7.0), torch.full((3, 3, 128, 128), float("nan"), device="cuda")
            p.linattn_forward(Q if queries else None, K, V, decay, O if queries else None, state_in=f32(d.S), state_out=S, offsets=off, max_len=200)
            assert np.array_equal(S.cpu().numpy(), d.S) and torch.all(O == -7.0)
        outs, dS = gradients(p, d, 0.5, 200)
        assert np.array_equal(dS.cpu().numpy(), d.dS) and all(torch.all(t == -7.0) for t in outs)
        assert p.status() == B.IKBO_OK
