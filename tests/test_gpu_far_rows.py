"""Linear attention, its reads, drafted trees and rotations with axes where elements lie 2^31 and more apart."""
import numpy as np
import pytest
import torch

import qcache_util as QC
from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_linattn import f32, i32, offsets_of, plan

pytestmark = pytest.mark.gpu

D, STEP = 128, 2**20  # elements from one row to the next: 2 MB


def rows(n, parts, width, seed):
    """`parts` tensors [n, width], as slices of rows STEP apart and as they are."""
    far = torch.empty(n * STEP, dtype=torch.bfloat16, device="cuda").view(n, STEP)
    g = torch.Generator(device="cuda").manual_seed(seed)
    near = [torch.randn((n, width), generator=g, device="cuda").bfloat16() for _ in range(parts)]
    for k, x in enumerate(near):
        far[:, k * width:(k + 1) * width] = x
    return far, near


@pytest.mark.parametrize("max_len", [8, 60, 300])
def test_rows_far_apart(max_len):
    """Past 2^31 elements, in every variant and both directions: bits as those of rows side by side."""
    H, n = 2, 2300
    far, near = rows(n, 8, H * D, max_len)
    view = lambda k: far[:, k * H * D:(k + 1) * H * D].unflatten(1, (H, D))  # noqa: E731
    lens = [max_len] * (n // max_len) + [n % max_len]
    off, decay = i32(offsets_of(lens)), f32([0.97, 1.0])
    x = [t.unflatten(1, (H, D)) for t in near]
    with plan() as p:
        states = []
        for get in (view, lambda k: x[k]):
            S, dS = (torch.full((len(lens), H, D, D), float("nan"), device="cuda") for _ in range(2))
            p.linattn_forward(get(0), get(1), get(2), decay, get(4), state_out=S, offsets=off, max_len=max_len)
            p.linattn_backward(get(0), get(1), get(2), get(3), decay, get(5), get(6), get(7), d_state_in=dS, offsets=off, max_len=max_len)
            states.append((S, dS))
        for k in range(4, 8):
            assert torch.equal(view(k), x[k])
        assert torch.equal(states[0][0], states[1][0]) and torch.equal(states[0][1], states[1][1])
        assert p.status() == B.IKBO_OK


def test_states_past_32_bits():
    """8192 users of 17 heads: 2.3 * 10^9 elements of states; one row each, products that are exact."""
    U, H = 8192, 17
    g = torch.Generator(device="cuda").manual_seed(0)
    Q, K, V, dO = (torch.randint(-2, 3, (U, H, D), generator=g, device="cuda").bfloat16() for _ in range(4))
    S, decay = torch.empty((U, H, D, D), device="cuda"), f32([0.5] * H)
    O, dQ, dK, dV = (torch.empty_like(Q) for _ in range(4))
    m = torch.arange(U, dtype=torch.int32, device="cuda").flip(0).contiguous()
    X = torch.randint(-2, 3, (U, H, 8, D), generator=g, device="cuda").bfloat16()
    with B.Plan(U, U, H) as p:
        p.linattn_forward(Q, K, V, decay, O, state_out=S, n_users=U, scale=1.0)
        for a in range(0, U, 512):
            b = slice(a, a + 512)
            assert torch.equal(S[b], K[b].float()[..., None] * V[b].float()[..., None, :]), a
        q, k, v, do = (t.double() for t in (Q, K, V, dO))
        assert torch.equal(O, ((q * k).sum(-1, keepdim=True) * v).bfloat16())
        Y, dS = torch.empty_like(X), torch.empty_like(S)
        p.plan(m, U, H, 8)
        p.linattn_read_forward(X, S, Y, scale=1.0)
        xk = (X.double() * k.flip(0)[:, :, None]).sum(-1, keepdim=True)
        assert torch.equal(Y, (xk * v.flip(0)[:, :, None]).bfloat16())
        p.linattn_read_backward(X, S, X, None, dS, scale=1.0)
        for a in range(0, U, 512):
            x = X.flip(0)[a:a + 512].float()
            assert torch.equal(dS[a:a + 512], x.transpose(2, 3) @ x), a
        # the gradient from states to states: decay (dS + q do^T) at the first row
        p.linattn_backward(Q, K, V, dO, decay, dQ, dK, dV, state_in=S, d_state_out=S, d_state_in=dS, n_users=U, scale=1.0)
        for a in range(0, U, 512):
            b = slice(a, a + 512)
            assert torch.equal(dS[b], 0.5 * (S[b] + Q[b].float()[..., None] * dO[b].float()[..., None, :])), a
        # dq = (decay S + k v^T) do, S = k v^T
        assert torch.equal(dQ, (1.5 * (v * do).sum(-1, keepdim=True) * k).bfloat16())
        assert p.status() == B.IKBO_OK


def test_drafts_far_apart():
    n, Lq, H = 40, 64, 2
    far, near = rows(n * Lq, 2, H * D, 1)
    K, V = (far[:, k * H * D:(k + 1) * H * D].unflatten(1, (H, D)).unflatten(0, (n, Lq)) for k in range(2))
    k, v = (t.view(n, Lq, H, D) for t in near)
    st = QC.Store(5, [50], H, 16)
    data, table, ln = st.cuda()
    q, m = torch.randn((n, H, Lq, D), device="cuda").bfloat16(), torch.zeros(n, dtype=torch.int32, device="cuda")
    with plan() as p:
        p.plan(m, 1, H, Lq)
        a, b = torch.empty_like(q), torch.empty_like(q)
        p.attn_qcache_tree_forward(q, data, 16, table, ln, K, V, None, a)
        p.attn_qcache_tree_forward(q, data, 16, table, ln, k, v, None, b)
        assert torch.equal(a, b) and p.status() == B.IKBO_OK


@pytest.mark.parametrize("d,rot", [(128, 64), (100, 30)])
def test_rotations_far_apart(d, rot):
    far, (x, y) = rows(2300, 2, d, d)
    X, Y = (far[:, k * d:(k + 1) * d][:, None, None] for k in range(2))
    start = torch.arange(2300, dtype=torch.int32, device="cuda")[:, None].expand(2300, 2).contiguous()
    with plan() as p:
        axes = B.Rope(rot, axes=[j % 2 for j in range(rot // 2)])
        for r, call in ((axes, lambda a, b: p.rope_axes_forward(axes, a, b, start=start)),
                        (B.Rope(rot), lambda a, b: p.rope_forward(B.Rope(rot), a, b, start=start[:, 0].contiguous()))):
            call(X, Y)
            call(x[:, None, None], y[:, None, None])
            assert torch.equal(Y, y[:, None, None])
        assert p.status() == B.IKBO_OK
