"""ikbo_attn_forward repeats bit for bit where Lq does not divide the 128-row
query tile (rows behind the tile's last candidate are not the caller's data)."""
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B
from broadcast_gemm_attention_gb300 import inputs as gen
from gpu_util import check_attn_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Lq", [24, 40, 72, 120])
def test_rows_behind_the_last_candidate_have_no_say(Lq):
    x = gen.make_attn("repeat", 77, n_cand=17, n_users=2, H=4, Lq=Lq, d=128, Lkv=500)
    Q, K, V = (t.cuda() for t in (x.Q * 3, x.K, x.V))
    m = x.map.cuda()
    outs = []
    with B.Plan(17, 2, 4) as p:
        p.plan(m, 2, 4, Lq)
        for k in range(4):
            O = torch.empty_like(Q)
            junk = torch.randn_like(K) * 30  # other launches leave other bytes in shared memory
            p.attn_forward(Q, junk, junk, None, O)
            p.attn_forward(Q, K, V, None, O)
            outs.append(O)
        assert p.status() == B.IKBO_OK
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    x.Q = x.Q * 3
    check_attn_all(outs[0], x)


def test_self_rows_behind_the_candidates_rows():
    """Lq = 24: 120 rows of a tile are candidates', a user's own tile has 128.  The last eight meet
    keys of scores far above all before: their reference has to move like any other row's."""
    H, Lq, Lq_u, Lkv, d = 2, 24, 128, 300, 128
    g = torch.Generator().manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    Q, Qu, K, V = bf(7, H, Lq, d), bf(2, H, Lq_u, d), bf(2, H, Lkv, d), bf(2, H, Lkv, d)
    Qu[:, :, 120:] = 0
    Qu[:, :, 120:, 5] = 40
    K[:, :, :, 5] = 0
    K[:, :, 200, 5] = 60  # 2400 / sqrt(128) * log2(e) = 306 in powers of two, in the second tile of keys
    m = torch.tensor([0, 1, 1, 0, 1, 1, 1], dtype=torch.int32, device="cuda")
    O, Ou = torch.empty_like(Q), torch.empty_like(Qu)
    with B.Plan(7, 2, H) as p:
        p.plan(m, 2, H, Lq)
        p.attn_self_target_forward(Q, Qu, K, V, None, O, Ou)
        assert p.status() == B.IKBO_OK
    S = (Qu.double() @ K.double().transpose(-1, -2)) / d ** 0.5
    ref = torch.softmax(S, -1) @ V.double()
    # P's rounding (2^-8, numerator and not the sum), O's, and the scores' error at |s| <= 212 (2^-16 of it, twice)
    big = torch.softmax(S, -1) @ V.double().abs()
    assert bool(((Ou.double() - ref).abs() <= big * (2.0 ** -8 + 2.0 ** -7) + ref.abs() * 2.0 ** -8).all())
