"""Drafted trees over every variant of the history's attention, users without a history among them."""
import numpy as np
import pytest

from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_tree import Case, plan

pytestmark = pytest.mark.gpu


# rows a user and K/V head, and the bound on the tokens: what the history's variant goes by
@pytest.mark.parametrize("n,H,H_kv,Lq,Lkv,launches", [(9, 1, 1, 8, 400, 1), (12, 4, 2, 64, 1_000_000, 1), (12, 8, 1, 24, 1_000_000, 1), (20, 4, 1, 128, 700, 2)],
                         ids=["registers", "tiles", "tiles_short", "decoded"])
def test_histories_of_every_variant(n, H, H_kv, Lq, Lkv, launches):
    m = (np.arange(n) % 3).astype(np.int32)
    c = Case(n + Lq, [300, 0, 41], m, H, H_kv, Lq, 16, branch=4)
    with plan() as p:
        before = p.launches()
        O, lse = c.run(p, Lkv=Lkv)
        assert p.launches() == before + 1 + launches + 1  # the plan, the history's, the drafts'
        c.check(O, lse)
        O2, _ = c.run(p, Lkv=Lkv, lse=False)
        assert np.array_equal(O2.float().cpu().numpy(), O.float().cpu().numpy())
        assert p.status() == B.IKBO_OK
