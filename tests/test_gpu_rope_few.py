"""Rotations off the 16-byte path: rows shared by more threads than a CTA has, by a part of one, and more rows than
run at a time.  Tolerances as test_gpu_rope.py derives them."""
import numpy as np
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B
from test_gpu_rope import DT, check

pytestmark = pytest.mark.gpu

# pieces of a row (rot / 2 + d - rot, or rot / 2 in place) from 1 to 511, rows from one to more than all CTAs take at a time
SIZES = [(1, 8, 1, 512, 2), (1, 3, 1, 512, 510), (2, 2, 1, 511, 256), (1, 1, 3, 260, 250), (5, 9, 7, 130, 130), (38, 1, 1, 500, 4),
         (153, 2, 1, 300, 90), (700, 1, 1, 129, 126), (3000, 1, 1, 70, 70), (21000, 1, 1, 35, 32), (1, 5, 21000, 6, 6)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n,H,L,d,rot", SIZES)
def test_rows_shared_by_any_number_of_threads(dt, n, H, L, d, rot):
    g = torch.Generator().manual_seed(n + d)
    x = torch.randn((n, H, L, d), generator=g).to(DT[dt]).cuda()
    start = torch.randint(-50, 5000, (n,), generator=g, dtype=torch.int32)
    freqs = B.ikbo_rope_frequencies(rot)
    with B.Plan(64, 64, 4) as p:
        for inter in (False, True):
            r = B.Rope(rot, freqs, interleaved=inter)
            wide = torch.full((n, H, L, d + 3), 7.0, dtype=x.dtype, device="cuda")  # (rows apart by an odd stride)
            y = wide[..., 1:d + 1]
            p.rope_forward(r, x, y, start=start.cuda())
            check(y, x, start.numpy()[:, None].astype(np.int64) + np.arange(L), freqs, inter)
            assert torch.all(wide[..., 0] == 7.0) and torch.all(wide[..., d + 1:] == 7.0)
            z = x.clone()
            p.rope_forward(r, z, z, start=start.cuda())
            assert torch.equal(z, y)
            axes = B.Rope(rot, freqs, interleaved=inter, axes=[j % 2 for j in range(rot // 2)], n_axes=2)
            place = torch.arange(L, dtype=torch.int32).cuda()[:, None].expand(L, 2).contiguous()
            z = torch.full_like(x, float("nan"))
            p.rope_axes_forward(axes, x, z, positions=place, start=start.cuda()[:, None].expand(n, 2).contiguous())
            assert torch.equal(z, y)
        assert p.status() == B.IKBO_OK
