"""A broadcast rotation reads start[map[i]]: its length is the planned request's
number of users.  Refused on the host, before any launch."""
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B


@pytest.mark.parametrize("call", ["rope_forward", "rope_backward"])
@pytest.mark.parametrize("n", [0, 2, 8])
def test_a_start_of_another_length_is_refused(call, n):
    """Too short (the kernel would read behind it), or a position per candidate."""
    p = B.Plan.__new__(B.Plan)  # as a plan of 8 candidates and 3 users is after plan(); no device needed
    p.handle, p._map, p._request = None, None, ((8, 2, 8), 3)
    x = torch.zeros(8, 2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="each of the plan's 3 users"):
        getattr(p, call)(None, x, x, start=torch.zeros(n, dtype=torch.int32), broadcast=True)


@pytest.mark.gpu
def test_on_a_plan():
    x = torch.randn(8, 2, 8, 128).to(torch.bfloat16).cuda()
    y, r = torch.full_like(x, 7.0), B.Rope(128)
    m = torch.tensor([2, 0, 0, 1, 2, 2, 1, 1], dtype=torch.int32, device="cuda")
    with B.Plan(8, 5, 2) as p:
        p.plan(m, 3, 2, 8)
        before = p.launches()
        for n in (2, 8):
            for call in (p.rope_forward, p.rope_backward):
                with pytest.raises(ValueError):
                    call(r, x, y, start=torch.zeros(n, dtype=torch.int32, device="cuda"), broadcast=True)
        assert p.launches() == before
        start = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
        p.rope_forward(r, x, y, start=start, broadcast=True)
        each = torch.empty_like(x)
        p.rope_forward(r, x, each, start=start[m.long()].contiguous())
        assert torch.equal(y, each) and p.status() == B.IKBO_OK
