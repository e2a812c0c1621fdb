"""The plan's status is read and cleared in the order of the stream it is asked on."""
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_status_goes_by_its_own_stream():
    """A side stream's errors are read, and cleared, while the default stream is busy with other work."""
    side = torch.cuda.Stream()
    bad = torch.tensor([0, 9, 1], dtype=torch.int32, device="cuda")
    with B.Plan(3, 2, 1) as p:
        p.plan(bad, 2)
        assert p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE
        torch.cuda.synchronize()
        torch.cuda._sleep(1_000_000_000)  # half a second
        busy = torch.cuda.Event()
        busy.record()
        codes = []
        for _ in range(50):
            p.plan(bad, 2, stream=side)
            codes.append(p.status(side))
            codes.append(p.status(side))
        still = not busy.query()
        assert codes == [B.IKBO_ERR_MAP_OUT_OF_RANGE, B.IKBO_OK] * 50
        assert still
        torch.cuda.synchronize()
