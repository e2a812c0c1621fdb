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
