"""Rotary positions on the GPU against the definition in 64 bits.

Tolerance, from what the kernel rounds: the half-turn argument of sincospi is a
24-bit float (2^-25 of a half turn, pi 2^-25 in the angle), sincospi is within
2 ulp (2^-23), the factor and two fp32 products and a sum add 3 * 2^-24; in all
under 6e-7 (|x| + |y|) |magnitude| for fp32.  16-bit types use the hardware's sine
and cosine, 2^-20.5 absolute (6.8e-7) instead of 2^-23, and an argument in
radians (pi 2^-24 more): under 1.5e-6.  Then half a step of the type.
"""
import numpy as np
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B
from qcache_util import rope_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(y, x, pos, freqs, inter, mag=1.0, backward=False):
    xd = x.double().cpu().numpy()
    ref = rope_ref(xd, pos, freqs, inter, mag, backward)
    rot = 2 * len(freqs)
    size = np.zeros_like(xd)
    h = rot // 2
    a, b = (xd[..., 0:rot:2], xd[..., 1:rot:2]) if inter else (xd[..., :h], xd[..., h:rot])
    both = np.abs(a) + np.abs(b)
    if inter:
        size[..., 0:rot:2] = size[..., 1:rot:2] = both
    else:
        size[..., :h] = size[..., h:rot] = both
    info = torch.finfo(y.dtype)
    bound = (6e-7 if y.dtype == torch.float32 else 1.5e-6) * abs(mag) * size + info.eps / 2 * np.abs(ref) + info.tiny * info.eps
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= bound), float(np.nanmax(np.abs(got - ref) - bound))
    assert np.array_equal(got[..., rot:], xd[..., rot:])


def plan():
    return B.Plan(64, 64, 4)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,H,L,d,rot", [(1, 1, 1, 2, 2), (1, 8, 1, 128, 128), (3, 5, 7, 80, 20), (2, 3, 33, 64, 32),
                                         (5, 2, 16, 128, 64), (2, 9, 3, 256, 256), (1, 1, 1, 512, 512), (4, 4, 5, 40, 16),
                                         (17, 1, 1, 96, 96), (2, 2, 3, 33, 30), (300, 2, 5, 72, 48)])
def test_against_the_definition(dt, inter, n, H, L, d, rot):
    g = torch.Generator().manual_seed(n * 1000 + d)
    x = torch.randn((n, H, L, d), generator=g).to(DT[dt]).cuda()
    start = torch.randint(-50, 5000, (n,), generator=g, dtype=torch.int32)
    freqs = B.ikbo_rope_frequencies(rot)
    r = B.Rope(rot, freqs, interleaved=inter, magnitude=1.25)
    pos = start.numpy()[:, None].astype(np.int64) + np.arange(L)
    with plan() as p:
        y = torch.full_like(x, float("nan"))
        p.rope_forward(r, x, y, start=start.cuda())
        check(y, x, pos, freqs, inter, 1.25)
        dx = torch.full_like(x, float("nan"))
        p.rope_backward(r, x, dx, start=start.cuda())
        check(dx, x, pos, freqs, inter, 1.25, backward=True)
        z = x.clone()
        p.rope_forward(r, z, z, start=start.cuda())  # in place
        assert torch.equal(z, y)
        assert p.status() == B.IKBO_OK and p.launches() == 3


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "turns"])
def test_far_positions(scaling):
    """Angles stay exact where a float product would have lost them."""
    freqs = B.ikbo_rope_frequencies(64, scaling=scaling, factor=8.0, original_len=8192.0, low_turns=1.0, high_turns=4.0)
    start = torch.tensor([0, 1, 999_983, 16_777_217, 2**31 - 1, -2**31], dtype=torch.int32)
    x = torch.randn(6, 2, 2, 64, generator=torch.Generator().manual_seed(1)).cuda()
    with plan() as p:
        y = torch.empty_like(x)
        p.rope_forward(B.Rope(64, freqs), x, y, start=start.cuda())
        # frequencies are doubles: their own rounding moves the farthest angle by 2^31 2^-53 = 2.4e-7 at most
        pos = start.numpy().astype(np.int64)[:, None] + np.arange(2)
        xd = x.double().cpu().numpy()
        ref = rope_ref(xd, pos, freqs)
        size = np.abs(xd[..., :32]) + np.abs(xd[..., 32:])
        bound = (6e-7 + 2.0 ** -22) * np.concatenate([size, size], -1) + 2.0 ** -24 * np.abs(ref)
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= bound)


def test_gradient_against_differences():
    """The forward is linear in X, so a difference of any size is its derivative."""
    freqs = B.ikbo_rope_frequencies(32)
    r = B.Rope(32, freqs, interleaved=True, magnitude=0.5)
    g = torch.Generator().manual_seed(2)
    x, e, dy = (torch.randn(4, 3, 5, 48, generator=g).cuda() for _ in range(3))
    start = torch.randint(0, 9999, (4,), generator=g, dtype=torch.int32).cuda()
    with plan() as p:
        y0, y1, dx = (torch.empty_like(x) for _ in range(3))
        p.rope_forward(r, x, y0, start=start)
        p.rope_forward(r, x + e, y1, start=start)
        p.rope_backward(r, dy, dx, start=start)
    left = ((y1 - y0).double() * dy.double()).sum().item()
    right = (dx.double() * e.double()).sum().item()
    scale = (e.double().abs() * dy.double().abs()).sum().item() * 4
    assert abs(left - right) <= 2e-6 * scale


def test_broadcast_takes_the_users_position():
    m = torch.tensor([2, 0, 0, 1, 2, 2, 5, -1], dtype=torch.int32)
    start = torch.tensor([10, 700, 123456], dtype=torch.int32)
    x = torch.randn(8, 2, 8, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    r = B.Rope(128)
    with B.Plan(8, 3, 2) as p:
        y = torch.full_like(x, 7.0)
        with pytest.raises(B.IkboError) as e:
            p.rope_forward(r, x, y, start=start.cuda(), broadcast=True)
        assert e.value.code == B.IKBO_ERR_NOT_PLANNED
        p.plan(m.cuda(), 3, 2, 8)
        assert p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE
        p.rope_forward(r, x, y, start=start.cuda(), broadcast=True)
        pos = start.numpy()[m.numpy()[:6]].astype(np.int64)[:, None] + np.arange(8)
        check(y[:6], x[:6], pos, B.ikbo_rope_frequencies(128), False)
        assert bool((y[6:] == 7.0).all())  # candidates without a user keep their rows
        assert p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE
        with pytest.raises(B.IkboError) as e:
            p.rope_forward(r, x[:4], y[:4], start=start.cuda(), broadcast=True)
        assert e.value.code == B.IKBO_ERR_INVALID_ARG


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_strided_slices_of_a_projection(dt):
    """Heads of a wider projection, [token][3 H d]; token-major and head-major views; an odd offset."""
    n, H, d = 37, 4, 32
    wide = torch.randn(n, 3 * H * d + 8, generator=torch.Generator().manual_seed(4)).to(DT[dt]).cuda()
    freqs = B.ikbo_rope_frequencies(32)
    r = B.Rope(32, freqs)
    start = torch.arange(n, dtype=torch.int32).cuda() * 3
    pos = (np.arange(n) * 3)[:, None]
    for off in (0, H * d, 8, 3):
        x = wide[:, off:off + H * d].view(n, H, d)
        out = torch.full((H, n, d + 2), 5.0, dtype=DT[dt], device="cuda")
        y = out.permute(1, 0, 2)[:, :, :d]
        with plan() as p:
            p.rope_forward(r, x, y, start=start)
        check(y[:, :, None, :], x[:, :, None, :], pos, freqs, False)
        assert bool((out[:, :, d:] == 5.0).all())
    # [1, H, n, d] of a token-major tensor: tokens at their own places, no start
    x = wide[:, :H * d].view(1, n, H, d).permute(0, 2, 1, 3)
    y = torch.empty((1, H, n, d), dtype=DT[dt], device="cuda")
    with plan() as p:
        p.rope_forward(r, x, y)
    check(y, x, np.arange(n)[None, :], freqs, False)


def test_in_place_leaves_the_rest_and_wrong_calls_are_refused():
    x = torch.randn(3, 2, 4, 64).to(torch.bfloat16).cuda()
    x[..., 32:] = float("nan")
    keep = x.clone()
    r = B.Rope(32)
    with plan() as p:
        p.rope_forward(r, x, x)
        assert torch.equal(x[..., 32:].view(torch.int16), keep[..., 32:].view(torch.int16))
        p.rope_forward(r, x[:0], x[:0])  # nothing to do
        assert p.launches() == 1
        for bad in (dict(X=x.cpu(), Y=x), dict(X=x, Y=x[:2]), dict(X=x, Y=x.float()), dict(X=x.long(), Y=x.long()),
                    dict(X=x[..., ::2], Y=x[..., ::2]), dict(X=x, Y=x, start=torch.zeros(2, dtype=torch.int32).cuda()),
                    dict(X=x, Y=x, start=torch.zeros(3).cuda()), dict(X=x[0, 0], Y=x[0, 0])):
            with pytest.raises(ValueError):
                p.rope_forward(r, bad["X"], bad["Y"], start=bad.get("start"))
        with pytest.raises(B.IkboError):
            p.rope_forward(B.Rope(128), x, x)


def test_infinities_and_nan_stay_in_their_pairs():
    x = torch.randn(2, 1, 1, 32).cuda()
    x[0, 0, 0, 3], x[1, 0, 0, 5] = float("inf"), float("nan")
    with plan() as p:
        y = torch.empty_like(x)
        p.rope_forward(B.Rope(32), x, y, start=torch.tensor([5, 6], dtype=torch.int32).cuda())
    bad = ~torch.isfinite(y[:, 0, 0])
    assert set(map(tuple, bad.nonzero().tolist())) == {(0, 3), (0, 19), (1, 5), (1, 21)}


def test_on_another_stream_and_in_a_graph():
    x = torch.randn(64, 4, 8, 128).to(torch.bfloat16).cuda()
    start = torch.arange(64, dtype=torch.int32).cuda()
    r = B.Rope(128)
    with plan() as p:
        y = torch.empty_like(x)
        p.rope_forward(r, x, y, start=start)
        z = torch.zeros_like(x)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        p.rope_forward(r, x, z, start=start, stream=s)
        s.synchronize()
        assert torch.equal(y, z)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.rope_forward(r, x, z, start=start)
        start.add_(1000)
        graph.replay()
        p.rope_forward(r, x, y, start=start)
        assert torch.equal(y, z)
