"""Refusals of the drafted trees' call: for their own reason also under capture, and before the plan's memory is touched."""
import pytest
import torch

import qcache_util as QC
from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu

INVALID, UNSUPPORTED, CUDA, NOT_PLANNED = 1, 2, 3, 6


def call(p, c, stream=None, **other):
    """The C entry without log-sum-exp, any of its arguments replaced; addresses of the case's tensors."""
    a = dict(p=p.handle, Q=c.q.data_ptr(), data=c.data.data_ptr(), n_pages=c.data.shape[0], page=c.st.page, H_kv=c.H_kv,
             table=c.table.data_ptr(), blocks=c.table.shape[1], lens=c.ln.data_ptr(), K=c.k.data_ptr(), V=c.v.data_ptr(),
             stride=c.H_kv * 128, parents=None, O=c.o.data_ptr(), lse=None, Lkv=100, d=128, scale=0.1, stream=stream)
    a.update(other)
    return B.load().ikbo_attn_qcache_tree_forward(*a.values())


class Call:
    def __init__(self):
        self.st, self.H_kv = QC.Store(3, [40], 2, 16), 2
        self.data, self.table, self.ln = self.st.cuda()
        self.q = torch.zeros((512, 16, 128, 128), dtype=torch.bfloat16, device="cuda")
        self.k, self.v = (torch.zeros((512, 128, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.o = torch.full_like(self.q, 3.0)
        self.map = torch.zeros(512, dtype=torch.int32, device="cuda")


BAD = [(dict(scale=0.0), INVALID), (dict(Lkv=0), INVALID), (dict(d=64), UNSUPPORTED), (dict(H_kv=3), INVALID), (dict(page=17), UNSUPPORTED),
       (dict(O=None), INVALID), (dict(lens=None), INVALID), (dict(lse=2), INVALID)]


def test_a_refused_call_allocates_nothing():
    c = Call()
    with B.Plan(512, 4, 16) as p:
        assert call(p, c) == NOT_PLANNED
        p.plan(c.map, 1, 16, 128)
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        for other, code in BAD:
            assert call(p, c, **other) == code, other
        assert torch.cuda.mem_get_info()[0] >= free  # (the log-sum-exp takes 4 MB)
        assert p.launches() == 1 and torch.all(c.o == 3.0) and p.status() == B.IKBO_OK


def test_a_refused_call_under_capture_says_why():
    c = Call()
    with B.Plan(512, 4, 16) as p:
        p.plan(c.map, 1, 16, 128)
        torch.cuda.synchronize()
        graph, codes = torch.cuda.CUDAGraph(), []
        x = torch.zeros(1, device="cuda")
        with torch.cuda.graph(graph):
            x += 1
            s = torch.cuda.current_stream().cuda_stream
            codes = [call(p, c, stream=s, **other) for other, _ in BAD]
            good = call(p, c, stream=s)  # that one would have to allocate
        assert codes == [code for _, code in BAD] and good == CUDA
        graph.replay()
        torch.cuda.synchronize()
        assert float(x) == 1.0 and torch.all(c.o == 3.0) and p.status() == B.IKBO_OK


def test_more_heads_than_a_grid_has_are_refused_before_any_launch():
    H = 65536
    st = QC.Store(4, [0], 1, 16)
    table, ln = st.cuda()[1:]
    data = torch.zeros((1, H, 1, 2560), dtype=torch.uint8, device="cuda")
    x = torch.zeros((1, H, 24, 128), dtype=torch.bfloat16, device="cuda")
    kv, o, m = torch.zeros((1, 24, H, 128), dtype=torch.bfloat16, device="cuda"), torch.full_like(x, 3.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    with B.Plan(1, 1, H) as p:
        p.plan(m, 1, H, 24)
        with pytest.raises(B.IkboError) as e:
            p.attn_qcache_tree_forward(x, data, 16, table, ln, kv, kv, None, o)
        assert e.value.code == UNSUPPORTED and p.launches() == 1
        torch.cuda.synchronize()
        assert torch.all(o == 3.0) and p.status() == B.IKBO_OK
