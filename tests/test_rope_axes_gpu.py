"""Rotary positions with several axes, and their gradient, on the GPU against 64-bit rotations
(bounds as in test_rope_gpu.py)."""
import pytest
import torch

from cache_reference import rotate

pytestmark = pytest.mark.gpu


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def _check(got, x, freq, pos, mult, interleaved):
    y, size = rotate(x.cpu(), freq.cpu(), pos, mult, interleaved)
    u = torch.finfo(got.dtype).eps / 2
    bound = u * y.abs() + size * 2.0 ** -20 + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    assert ((got.cpu().double() - y).abs() - bound).max().item() <= 0


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("D,sections", [(128, (16, 24, 24)), (128, (16, 16)), (80, (20, 20)), (64, (1, 2, 3, 4)), (96, (48,)),
                                        (66, (10, 0, 7)), (33, (5, 5)), (512, (128, 128))])
@pytest.mark.parametrize("mixed", [False, True])
def test_axes(io, interleaved, inverse, D, sections, mixed):
    sdpa = _sdpa()
    B, Hq, Hkv, S = 2, 5, 2, 37
    g = torch.Generator().manual_seed(D + len(sections))
    q, k = (torch.randn(B, S, H, D, generator=g).to(io).cuda().transpose(1, 2) for H in (Hq, Hkv))
    axes = sdpa.rope_axes(sections, mixed=mixed)
    assert sorted(axes.tolist()) == [a for a, n in enumerate(sections) for _ in range(n)]
    freq = sdpa.rope_inv_freq(2 * sum(sections))
    positions = torch.randint(-100, 100000, (len(sections), B, S), generator=g, dtype=torch.int32)
    fn = sdpa.rope_bwd if inverse else sdpa.rope_fwd
    got = fn(q, k, freq, positions=positions.cuda(), axes=axes, interleaved=interleaved, mult=1.5)
    pos = positions.long()[axes.cpu().long()].permute(1, 2, 0) * (-1 if inverse else 1)
    for y, x in zip(got, (q, k)):
        _check(y, x, freq, pos, 1.5, interleaved)


def test_one_axis_is_the_plain_rotation():
    sdpa = _sdpa()
    q = torch.randn(2, 4, 50, 128).bfloat16().cuda()
    freq, positions = sdpa.rope_inv_freq(128), torch.randint(0, 9999, (2, 50), dtype=torch.int32).cuda()
    a = sdpa.rope_fwd(q, None, freq, positions=positions)[0]
    b = sdpa.rope_fwd(q, None, freq, positions=positions[None], axes=sdpa.rope_axes((64,)))[0]
    assert torch.equal(a, b)
    # every axis at the same positions, shared by the batch rows
    c = sdpa.rope_fwd(q, None, freq, positions=positions[:1].expand(3, 50).contiguous(), axes=sdpa.rope_axes((16, 24, 24)))[0]
    assert torch.equal(c[0], a[0])


def test_axes_outside_count_as_the_nearest():
    sdpa = _sdpa()
    q = torch.randn(1, 2, 9, 32).bfloat16().cuda()
    freq, positions = sdpa.rope_inv_freq(32), torch.randint(0, 99, (2, 9), dtype=torch.int32).cuda()
    odd = torch.tensor([-5, 0, 1, 2, 99, -(1 << 31), (1 << 31) - 1, 0] * 2, dtype=torch.int32).cuda()
    for interleaved in (False, True):
        a = sdpa.rope_fwd(q, None, freq, positions=positions, axes=odd, interleaved=interleaved)[0]
        assert torch.equal(a, sdpa.rope_fwd(q, None, freq, positions=positions, axes=odd.clamp(0, 1), interleaved=interleaved)[0])


def test_gradient_is_the_transposed_map():
    """<y, R x> = <R^T y, x> in 64 bits of the fp32 outputs' neighbours: the rounding of each side is 2^-9 of
    its terms, bf16; and R^T R = mult^2."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(1)
    x, y = (torch.randn(1, 1, 200, 64, generator=g).bfloat16().cuda() for _ in range(2))
    freq, axes = sdpa.rope_inv_freq(64), sdpa.rope_axes((8, 12, 12), mixed=True)
    positions = torch.randint(0, 5000, (3, 200), generator=g, dtype=torch.int32).cuda()
    kw = dict(positions=positions, axes=axes)
    rx, ry = sdpa.rope_fwd(x, None, freq, **kw)[0], sdpa.rope_bwd(y, None, freq, **kw)[0]
    a, b = y.double() * rx.double(), ry.double() * x.double()
    assert abs((a.sum() - b.sum()).item()) <= 2.0 ** -8 * (a.abs().sum() + b.abs().sum()).item() + 2.0 ** -18 * 64 * 200
    back = sdpa.rope_bwd(rx, None, freq, **kw)[0]
    # two roundings to bf16, each at most 2^-8 of a pair's length
    length = (x.double()[..., :32].square() + x.double()[..., 32:].square()).sqrt().repeat(1, 1, 1, 2)
    assert ((back.double() - x.double()).abs() <= 2.0 ** -6 * length + 2.0 ** -30).all()
