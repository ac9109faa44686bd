"""The rotary embedding and its gradient on the GPU against 64-bit rotations.

Bounds. With c, s the exact cosine and sine: the angle carries 2^-25 of itself in
half turns (at most pi * 2^-25 radians), sincospif and the factor a few units, so each
of c and s is off by at most 2^-21; the two products and their sum round to fp32
(2^-23 of |a| + |b|), and the result once to the io type: for each element
  |got - exact| <= u |exact| + mult (|a| + |b|) 2^-20,   u = finfo.eps / 2
(plus 2^-25 where fp16 results are subnormal). Columns that pass through are equal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def _exact(x, f, pos, mult, interleaved, inverse):
    """(rotated x, |a| + |b| at each rotated column) for x (B, H, S, D) in fp64, pos (B, S)."""
    rot = 2 * f.numel()
    x = x.double()
    angle = pos.double()[:, None, :, None] * f.double()
    c, s = torch.cos(angle) * mult, torch.sin(angle) * mult * (-1 if inverse else 1)
    y, size = x.clone(), torch.zeros_like(x)
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mult)
    return y, size


def _close(name, got, x, f, pos, mult, interleaved, inverse):
    y, size = _exact(x.cpu(), f.cpu(), pos.cpu(), mult, interleaved, inverse)
    rot = 2 * f.numel()
    got = got.cpu()
    assert torch.equal(got[..., rot:], x.cpu()[..., rot:]), f"{name}: columns past rot_dim changed"
    u = torch.finfo(got.dtype).eps / 2
    bound = u * y.abs() + size * 2.0 ** -20 + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    over = ((got.double() - y).abs() - bound).max().item() if got.numel() else -1.0
    assert over <= 0, f"{name}: {over:.3e} over its bound"


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 16), (80, 32), (80, 48), (256, 256), (72, 72), (64, 20),
                                   (8, 2), (9, 4), (33, 32), (512, 512), (80, 20), (80, 40), (96, 24), (96, 48),
                                   (88, 80), (10, 4)])
def test_rotation(io, interleaved, inverse, D, rot):
    sdpa = _sdpa()
    B, Hq, Hkv, S = 2, 6, 3, 37
    g = torch.Generator().manual_seed(D + rot)
    q, k = (torch.randn(B, H, S, D, generator=g).to(io).cuda() for H in (Hq, Hkv))
    f = sdpa.rope_inv_freq(rot)
    fn = sdpa.rope_bwd if inverse else sdpa.rope_fwd
    got = fn(q, k, f, interleaved=interleaved, offset=5, mult=1.25)
    pos = (torch.arange(S) + 5).expand(B, S)
    for name, y, x in (("q", got[0], q), ("k", got[1], k)):
        assert y.is_contiguous()
        _close(name, y, x, f, pos, 1.25, interleaved, inverse)


@pytest.mark.parametrize("B,S,Hq,Hkv", [(1, 1, 1, 0), (16, 1, 32, 8), (1, 4099, 1, 1), (3, 65, 5, 5), (2, 300, 41, 1)])
def test_sizes_and_heads(B, S, Hq, Hkv):
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(S)
    q = torch.randn(B, Hq, S, 128, generator=g).bfloat16().cuda()
    k = torch.randn(B, Hkv, S, 128, generator=g).bfloat16().cuda() if Hkv else None
    f = sdpa.rope_inv_freq(128)
    yq, yk = sdpa.rope_fwd(q, k, f)
    pos = torch.arange(S).expand(B, S)
    _close("q", yq, q, f, pos, 1.0, False, False)
    if Hkv:
        _close("k", yk, k, f, pos, 1.0, False, False)
    else:
        assert yk is None


@pytest.mark.parametrize("start", [0, 1 << 17, 1 << 24, (1 << 31) - 50])
def test_far_positions(start):
    """Angles keep their value at every position that an int32 holds: the exact angle is
    taken with integer arithmetic on the fp64 frequency."""
    from fractions import Fraction
    sdpa = _sdpa()
    f = sdpa.rope_inv_freq(64)
    x = torch.zeros(1, 1, 50, 64).bfloat16().cuda()
    x[..., :32] = 1.0  # the result is (cos, sin)
    got = sdpa.rope_fwd(x, None, f, offset=start)[0].cpu().double()
    # 2 pi to 40 digits, so that the angle modulo a turn is exact far beyond fp64
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750")
    for s in (0, 1, 49):
        for i in (0, 1, 7, 31):
            turns = Fraction(start + s) * Fraction(f[i].item()) / two_pi
            a = float((turns - math.floor(turns)) * two_pi)
            # the frequency's own rounding to a fraction of a turn: position * 2^-53 turns
            tol = 2.0 ** -8 + 2.0 ** -20 + (start + s) * 2.0 ** -53 * 2 * math.pi
            assert abs(got[0, 0, s, i] - math.cos(a)) <= tol
            assert abs(got[0, 0, s, 32 + i] - math.sin(a)) <= tol


@pytest.mark.parametrize("shape", ["(S,)", "(B, S)"])
def test_positions(shape):
    sdpa = _sdpa()
    B, S = 3, 130
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-1000, 100000, (S,) if shape == "(S,)" else (B, S), generator=g, dtype=torch.int32)
    q = torch.randn(B, 4, S, 64, generator=g).half().cuda()
    f = sdpa.rope_inv_freq(64, 500000.0)
    got = sdpa.rope_fwd(q, None, f, positions=pos.cuda())[0]
    _close("q", got, q, f, pos.expand(B, S), 1.0, False, False)


@pytest.mark.parametrize("D,rot", [(128, 128), (80, 40)])
def test_strides_and_in_place(D, rot):
    """A fused (B, S, H, D) projection: rotated out of it, back into it, and within it."""
    sdpa = _sdpa()
    B, S, Hq, Hkv = 2, 77, 4, 2
    g = torch.Generator().manual_seed(2)
    fused = torch.randn(B, S, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    q, k = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hkv].transpose(1, 2)
    f = sdpa.rope_inv_freq(rot)
    pos = torch.arange(S).expand(B, S)
    yq, yk = sdpa.rope_fwd(q, k, f)
    _close("q", yq, q, f, pos, 1.0, False, False)
    _close("k", yk, k, f, pos, 1.0, False, False)
    back = torch.full_like(fused, math.nan)
    sdpa.rope_fwd(q, k, f, q_out=back[:, :, :Hq].transpose(1, 2), k_out=back[:, :, Hq:Hq + Hkv].transpose(1, 2))
    assert torch.equal(back[:, :, :Hq].transpose(1, 2), yq) and torch.equal(back[:, :, Hq:Hq + Hkv].transpose(1, 2), yk)
    assert torch.isnan(back[:, :, Hq + Hkv:]).all()  # the values' place is not touched
    values = fused[:, :, Hq + Hkv:].clone()
    sdpa.rope_fwd(q, k, f, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(fused[:, :, Hq + Hkv:], values)
    # rows that start off a 16-byte boundary, and heads that share one input row
    odd = torch.randn(B, 3, S, D + 1, generator=g).bfloat16().cuda()[..., 1:]
    _close("odd", sdpa.rope_fwd(odd, None, f)[0], odd, f, pos, 1.0, False, False)
    wide = torch.randn(B, 1, S, D, generator=g).bfloat16().cuda().expand(B, 3, S, D)
    _close("broadcast", sdpa.rope_fwd(wide, None, f)[0], wide, f, pos, 1.0, False, False)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_off_their_alignment(shift, interleaved):
    """Rows that start 2, 4 or 8 bytes past a 16-byte boundary, in or out."""
    sdpa = _sdpa()
    B, H, S, D = 2, 3, 33, 64
    g = torch.Generator().manual_seed(shift)
    f = sdpa.rope_inv_freq(32)
    pos = torch.arange(S).expand(B, S)
    x = torch.randn(B, H, S, D + 8, generator=g).half().cuda()[..., shift:shift + D]
    _close("in", sdpa.rope_fwd(x, None, f, interleaved=interleaved)[0], x, f, pos, 1.0, interleaved, False)
    room = torch.full((B, H, S, D + 8), math.nan, dtype=torch.half, device="cuda")
    y = room[..., shift:shift + D]
    sdpa.rope_fwd(x.contiguous(), None, f, interleaved=interleaved, q_out=y)
    _close("out", y, x, f, pos, 1.0, interleaved, False)
    assert torch.isnan(room[..., :shift]).all() and torch.isnan(room[..., shift + D:]).all()


def test_no_rows():
    sdpa = _sdpa()
    f = sdpa.rope_inv_freq(64)
    q = torch.zeros(2, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    yq, yk = sdpa.rope_fwd(q, q[:, :2], f)
    assert yq.shape == q.shape and yk.shape == (2, 2, 0, 64)


def test_gradient_is_the_transposed_map():
    """<rope(x), g> = <x, rope_bwd(g)>: in fp64 up to the two roundings to fp16, each at
    most 2^-11 of the products' magnitudes."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(3)
    x, y = (torch.randn(2, 3, 50, 96, generator=g).half().cuda() for _ in range(2))
    for scaling in ("none", "linear", "ntk", "bands"):
        f = sdpa.rope_inv_freq(64, scaling=scaling, factor=4.0, original_len=2048)
        for inter in (False, True):
            a = sdpa.rope_fwd(x, None, f, interleaved=inter, mult=1.1)[0].double()
            b = sdpa.rope_bwd(y, None, f, interleaved=inter, mult=1.1)[0].double()
            p, r = a * y.double(), x.double() * b
            tol = (2.0 ** -11 + 2.0 ** -18) * (p.abs().sum() + r.abs().sum())
            assert (p.sum() - r.sum()).abs() <= tol


def test_captured_and_on_another_stream():
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(2, H, 64, 128, generator=g).bfloat16().cuda() for H in (8, 2))
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    f = sdpa.rope_inv_freq(128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yq, yk = sdpa.rope_fwd(q, k, f, positions=pos)
    for start in (0, 1000):
        pos.copy_(torch.arange(start, start + 64))
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        want = sdpa.rope_fwd(q, k, f, offset=start, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])


def test_keys_alone():
    """No query heads: the keys are rotated all the same."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(6)
    k = torch.randn(2, 3, 50, 64, generator=g).bfloat16().cuda()
    f = sdpa.rope_inv_freq(64)
    for fn, inverse in ((sdpa.rope_fwd, False), (sdpa.rope_bwd, True)):
        out = torch.full_like(k, math.nan)
        yq, yk = fn(k[:, :0], k, f, k_out=out, offset=9)
        assert yq.shape == (2, 0, 50, 64) and yk is out
        _close("k", yk, k, f, (torch.arange(50) + 9).expand(2, 50), 1.0, False, inverse)
    for q, k in ((k[:, :0], k[:, :0]), (k[:, :0], None), (k[:0], k[:0])):  # nothing to rotate
        yq, yk = sdpa.rope_fwd(q, k, f)
        assert yq.shape == q.shape and (yk is None if k is None else yk.shape == k.shape)


@pytest.mark.parametrize("layout", ["(B, S, H, D)", "(B, H, S, D)"])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_neighbouring_slices_of_one_buffer(layout, Hkv):
    """Outputs beside their inputs in one buffer: every slice is written alone, in place or not."""
    sdpa = _sdpa()
    B, S, Hq, D = 2, 29, 4, 64
    g = torch.Generator().manual_seed(7)
    room = torch.randn(B, S, 2 * (Hq + Hkv), D, generator=g).bfloat16().cuda()
    if layout == "(B, H, S, D)":
        room = room.transpose(1, 2).contiguous().transpose(1, 2)
    f = sdpa.rope_inv_freq(D)
    cut = (0, Hq, Hq + Hkv, 2 * Hq + Hkv, 2 * (Hq + Hkv))
    q, k, yq, yk = (room[:, :, a:b].transpose(1, 2) for a, b in zip(cut, cut[1:]))
    want = sdpa.rope_fwd(q, k, f)
    x = room.clone()
    sdpa.rope_fwd(q, k, f, q_out=yq, k_out=yk)
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1]) and torch.equal(room[:, :, :Hq + Hkv], x[:, :, :Hq + Hkv])
    sdpa.rope_fwd(q, k, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    before = room.clone()
    for bad in (dict(q_out=yq, k_out=yq[:, :Hkv]), dict(q_out=q, k_out=q[:, :Hkv]), dict(q_out=yq, k_out=q[:, 1:1 + Hkv])):
        with pytest.raises(sdpa.SdpaError):
            sdpa.rope_fwd(q, k, f, **bad)
        assert torch.equal(room, before)
