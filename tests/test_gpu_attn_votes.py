"""Rows of a query tile that no load writes have no influence on the others: the
attention forward's results depend neither on what earlier launches left in
shared memory nor on the other users whose units ran on the same SM."""
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu

D = 128


def bf(g, *shape, big=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * big).to(torch.bfloat16)


def check(O, Q, K, V):
    """Q, O [users, H, rows, 128] against the definition: P's rounding (2^-8, in the numerator and not in
    the sum), O's, and the scores' fp32 error (2^-16 of sum |q k|, here below 2^-9, twice)."""
    S = (Q.double() @ K.double().transpose(-1, -2)) / D ** 0.5
    P = torch.softmax(S, -1)
    ref, mass = P @ V.double(), P @ V.double().abs()
    assert bool(((O.double() - ref).abs() <= mass * (2.0 ** -8 + 2.0 ** -8) + ref.abs() * 2.0 ** -8).all())


@pytest.mark.parametrize("Lq_u", [8, 40, 72, 136])
@pytest.mark.parametrize("candidates", [False, True])
def test_users_own_rows_repeat(Lq_u, candidates):
    """Tiles of the users' own queries that fill part of 128 rows, the first on their CTA; between
    the calls other launches leave other bytes there."""
    H, Lq, Lkv, U = 4, 32, 500, 3
    g = torch.Generator(device="cuda").manual_seed(Lq_u)
    Qu, K, V = bf(g, U, H, Lq_u, D, big=3.0), bf(g, U, H, Lkv, D), bf(g, U, H, Lkv, D)
    m = torch.tensor([2, 0, 1, 2, 0], dtype=torch.int32, device="cuda")
    Q = bf(g, 5, H, Lq, D, big=3.0)
    # junk that fills the SMs: 64 users' tiles of 128 rows
    jm = torch.arange(64 * 4, dtype=torch.int32, device="cuda") // 4
    jQ = bf(g, 256, H, Lq, D)
    outs = []
    with B.Plan(5, U, H) as p, B.Plan(256, 64, H) as junk:
        p.plan(m, U, H, Lq)
        junk.plan(jm, 64, H, Lq)
        for k in range(4):
            jK = bf(g, 64, H, 130, D, big=30.0)
            junk.attn_forward(jQ, jK, jK, None, torch.empty_like(jQ))
            Ou = torch.empty_like(Qu)
            if candidates:
                O = torch.empty_like(Q)
                p.attn_self_target_forward(Q, Qu, K, V, None, O, Ou)
            else:
                p.attn_self_target_forward(None, Qu, K, V, None, None, Ou)
            outs.append(Ou)
        assert p.status() == B.IKBO_OK and junk.status() == B.IKBO_OK
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    check(outs[0], Qu, K, V)


@pytest.mark.parametrize("own", [False, True])
def test_other_users_have_no_say(own):
    """800 units, five or six to a CTA: with the first half of the users' keys, values and queries
    replaced, the others' rows are the same bit for bit."""
    H, U, Lkv = 8, 100, 300
    Lq = 40 if own else 24
    g = torch.Generator(device="cuda").manual_seed(5)
    n = U if own else 5 * U  # five candidates of 24 rows fill 120 rows of a tile
    m = torch.arange(5 * U, dtype=torch.int32, device="cuda") // 5
    Q, K, V = bf(g, n, H, Lq, D, big=3.0), bf(g, U, H, Lkv, D), bf(g, U, H, Lkv, D)
    outs = []
    with B.Plan(5 * U, U, H) as p:
        p.plan(m, U, H, 24)
        for k in range(3):
            O = torch.empty_like(Q)
            if own:
                p.attn_self_target_forward(None, Q, K, V, None, None, O)
            else:
                p.attn_forward(Q, K, V, None, O)
            outs.append(O[n * 6 // 10:].clone())
            if k == 0:
                check(O if own else O.view(U, 5, H, Lq, D).transpose(1, 2).reshape(U, H, 5 * Lq, D),
                      Q if own else Q.view(U, 5, H, Lq, D).transpose(1, 2).reshape(U, H, 5 * Lq, D), K, V)
            Q[:n // 2] = bf(g, n // 2, H, Lq, D)
            K[:U // 2] = bf(g, U // 2, H, Lkv, D)
            V[:U // 2] = bf(g, U // 2, H, Lkv, D, big=30.0)
        assert p.status() == B.IKBO_OK
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
