"""Rotary positions with several axes against the definition in 64 bits; tolerances as
test_gpu_rope.py derives them."""
import numpy as np
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def ref(x, pos, freqs, axes, inter, mag, backward):
    """x [n, H, L, d], pos [n, L, axes]; the size that errors scale with beside it."""
    half, y, size = len(freqs), np.array(x), np.zeros_like(x)
    for j, f in enumerate(freqs):
        a = (pos[..., axes[j]] * f)[:, None, :]
        c, s = np.cos(a) * mag, np.sin(a) * mag * (-1 if backward else 1)
        i, k = (2 * j, 2 * j + 1) if inter else (j, j + half)
        y[..., i] = x[..., i] * c - x[..., k] * s
        y[..., k] = x[..., k] * c + x[..., i] * s
        size[..., i] = size[..., k] = np.abs(x[..., i]) + np.abs(x[..., k])
    return y, size


def check(y, x, pos, freqs, axes, inter, mag=1.0, backward=False):
    want, size = ref(x.double().cpu().numpy(), pos, freqs, axes, inter, mag, backward)
    info = torch.finfo(y.dtype)
    bound = (6e-7 if y.dtype == torch.float32 else 1.5e-6) * abs(mag) * size + info.eps / 2 * np.abs(want) + info.tiny * info.eps
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) - bound))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n,H,L,d,rot,axes,inter,shared", [
    (1, 1, 1, 2, 2, 1, False, False), (3, 5, 7, 80, 20, 3, True, False), (2, 3, 33, 64, 32, 2, False, True),
    (5, 2, 16, 128, 128, 3, False, True), (4, 8, 9, 128, 96, 4, True, False), (2, 1, 3, 256, 256, 4, False, False),
    (300, 2, 1, 72, 48, 2, True, False), (6, 2, 4, 33, 30, 3, False, True)])
def test_against_the_definition(dt, n, H, L, d, rot, axes, inter, shared):
    g = torch.Generator().manual_seed(n * 1000 + d)
    x = torch.randn((n, H, L, d), generator=g).to(DT[dt]).cuda()
    start = torch.randint(-50, 5000, (n, axes), generator=g, dtype=torch.int32)
    place = torch.randint(-20, 60, (L, axes) if shared else (n, L, axes), generator=g, dtype=torch.int32)
    of = [j % axes for j in range(rot // 2)]
    freqs = B.ikbo_rope_frequencies(rot)
    r = B.Rope(rot, freqs, interleaved=inter, magnitude=1.25, axes=of, n_axes=axes)
    pos = start.numpy()[:, None].astype(np.float64) + place.numpy()
    with B.Plan(64, 64, 4) as p:
        for call, back in ((p.rope_axes_forward, False), (p.rope_axes_backward, True)):
            y = torch.full_like(x, float("nan"))
            call(r, x, y, positions=place.cuda(), start=start.cuda())
            check(y, x, pos, freqs, of, inter, 1.25, back)
            z = x.clone()
            call(r, z, z, positions=place.cuda(), start=start.cuda())  # in place
            assert torch.equal(y, z)
        y = torch.empty_like(x)
        p.rope_axes_forward(r, x, y, start=start.cuda())
        check(y, x, start.numpy()[:, None].repeat(L, 1).astype(np.float64), freqs, of, inter, 1.25)
        p.rope_axes_forward(r, x, y, positions=place.cuda())
        check(y, x, np.broadcast_to(place.numpy(), pos.shape).astype(np.float64), freqs, of, inter, 1.25)
        p.rope_axes_forward(r, x, y)
        check(y, x, np.zeros(pos.shape), freqs, of, inter, 1.25)


def test_one_axis_is_the_plain_rotation():
    x = torch.randn(7, 3, 5, 64, generator=torch.Generator().manual_seed(0)).cuda()
    start = torch.arange(7, dtype=torch.int32).cuda() * 1_000_003
    place = torch.arange(5, dtype=torch.int32).cuda()[:, None].contiguous()
    with B.Plan(64, 64, 4) as p:
        a, b = torch.empty_like(x), torch.empty_like(x)
        p.rope_forward(B.Rope(64), x, a, start=start)
        p.rope_axes_forward(B.Rope(64, axes=[0] * 32), x, b, positions=place, start=start[:, None].contiguous())
        assert torch.equal(a, b)


def test_the_sum_of_far_places_is_exact():
    """A start and a place whose sum passes 32 bits; the angle is the exact sum's."""
    x = torch.randn(2, 1, 1, 32, generator=torch.Generator().manual_seed(1)).cuda()
    start = torch.tensor([[2**31 - 1, -2**31], [2**31 - 1, 5]], dtype=torch.int32)
    place = torch.tensor([[2**31 - 1, -2**31]], dtype=torch.int32)
    pos = start.numpy()[:, None].astype(np.int64) + place.numpy().astype(np.int64)
    freqs = [2.0 ** -j for j in range(16)]
    of = [0] * 8 + [1] * 8
    with B.Plan(8, 8, 1) as p:
        y = torch.empty_like(x)
        p.rope_axes_forward(B.Rope(32, freqs, axes=of), x, y, positions=place.cuda(), start=start.cuda())
    # whole turns leave before 64-bit floats lose bits (angles below are then within 2^-50 of 2^32 radians, 4e-6: too coarse),
    # so the reference takes the remainder in extended precision
    two_pi = 2 * np.longdouble(np.pi) + np.longdouble(2.4492935982947064e-16)
    xd, want = x.double().cpu().numpy(), x.double().cpu().numpy().copy()
    for j, f in enumerate(freqs):
        t = pos[..., of[j]].astype(np.longdouble) * (np.longdouble(f) / two_pi)
        a = ((t - np.floor(t)) * 2 * np.pi).astype(np.float64)[:, None, :]
        want[..., j] = xd[..., j] * np.cos(a) - xd[..., j + 16] * np.sin(a)
        want[..., j + 16] = xd[..., j + 16] * np.cos(a) + xd[..., j] * np.sin(a)
    size = np.abs(xd[..., :16]) + np.abs(xd[..., 16:])
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= 7e-7 * np.concatenate([size, size], -1) + 2.0 ** -24 * np.abs(want))


def test_candidates_take_their_user_s_places():
    g = torch.Generator().manual_seed(3)
    m = torch.tensor([2, 0, 2, 1, 0, 9], dtype=torch.int32).cuda()
    x = torch.randn((6, 2, 8, 64), generator=g).cuda()
    start = torch.randint(0, 1000, (3, 2), generator=g, dtype=torch.int32)
    place = torch.randint(0, 20, (6, 8, 2), generator=g, dtype=torch.int32)
    of, freqs = [j % 2 for j in range(32)], B.ikbo_rope_frequencies(64)
    with B.Plan(64, 64, 4) as p:
        p.plan(m, 3, 2, 8)
        y = torch.full_like(x, -7.0)
        p.rope_axes_forward(B.Rope(64, freqs, axes=of), x, y, positions=place.cuda(), start=start.cuda(), broadcast=True)
        pos = start.numpy()[m.cpu().numpy()[:5]][:, None].astype(np.float64) + place.numpy()[:5]
        check(y[:5], x[:5], pos, freqs, of, False)
        assert torch.all(y[5] == -7.0) and p.status() == B.IKBO_ERR_MAP_OUT_OF_RANGE
        r = B.Rope(64, freqs, axes=of)
        with pytest.raises(ValueError):
            p.rope_axes_forward(r, x, y, start=start[:2].cuda(), broadcast=True)
        with pytest.raises(ValueError):
            p.rope_axes_forward(r, x, y, start=start.cuda())  # not one for each candidate
        with pytest.raises(ValueError):
            p.rope_axes_forward(r, x, y, positions=place[:, :7].cuda())
        with pytest.raises(ValueError):
            p.rope_axes_forward(B.Rope(64), x, y)
        with pytest.raises(B.IkboError):
            p.rope_forward(r, x, y)


def test_strides():
    """Slices of a wider projection, in and out, and rows of [rows, H, d] with places of their own."""
    g = torch.Generator().manual_seed(4)
    wide = torch.randn((9, 3, 4, 64), generator=g).to(torch.bfloat16).cuda()
    place = torch.randint(0, 5000, (9, 3), generator=g, dtype=torch.int32).cuda()
    r = B.Rope(48, axes=[j // 8 for j in range(24)])
    with B.Plan(8, 8, 1) as p:
        out = torch.zeros_like(wide)
        p.rope_axes_forward(r, wide[:, 1], out[:, 2], positions=place)
        plain = torch.empty((9, 4, 64), dtype=torch.bfloat16, device="cuda")
        p.rope_axes_forward(r, wide[:, 1].contiguous(), plain, positions=place)
        assert torch.equal(out[:, 2], plain) and not out[:, :2].any()
