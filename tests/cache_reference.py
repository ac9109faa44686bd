"""64-bit reference of the paged cache: rotations, 8-bit codes and scales, appending and
reading back, on the CPU, and the bounds that the tests hold the library to.

Bounds of a cached element. A rotated key in fp32 is off by at most 2^-20 (|a| + |b|) mult (the
angle 2^-25 of itself in half turns, sine and cosine a few units, two products and a sum); values are
taken as they are. One rounding follows: bf16 and fp16 finfo.eps / 2 of the value, fp16 below
2^-14 half of 2^-24; a code 2^-4 of the value, or half of the smallest step, 2^-10 of the scale."""
import math

import torch


def code(x):
    """x (fp64) to the nearest e4m3 value, ties to even, saturating at 448; NaN stays."""
    size = x.abs().clamp(max=448.0)
    _, e = torch.frexp(size.clamp(min=2.0 ** -6))
    step = torch.pow(torch.full_like(size, 2.0), (e - 4).double())
    return torch.copysign(torch.round(size / step) * step, x)


def scale_for(largest: float) -> float:
    """The smallest power of two, at least 2^-64, that brings `largest` within 448."""
    e = -64
    if largest > 0:
        m, e = math.frexp(largest / 448.0)
        e = max(e - 1 if m == 0.5 else e, -64)
    return 2.0 ** e


def rotate(x, freq, pos, mult=1.0, interleaved=False):
    """(x (B, H, S, D) turned by pos (B, S, pairs) * freq, |a| + |b| at each rotated column), fp64 CPU."""
    x = x.double()
    size = torch.zeros_like(x)
    if freq is None:
        return x, size
    n = freq.numel()
    angle = (pos.double() * freq.double())[:, None]
    c, s = angle.cos() * mult, angle.sin() * mult
    ia = torch.arange(0, 2 * n, 2) if interleaved else torch.arange(n)
    ib = ia + 1 if interleaved else ia + n
    y = x.clone()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mult)
    return y, size


def positions_of(lens, new, S, pairs, positions=None, axes=None):
    """(B, S, pairs) positions of every row of a call."""
    B = len(lens)
    if axes is not None:
        p = positions.long() if positions.dim() == 3 else positions.long()[:, None].expand(-1, B, -1)
        return p[axes.long()].permute(1, 2, 0)
    if positions is not None:
        p = positions.long() if positions.dim() == 2 else positions.long()[None].expand(B, -1)
        return p[..., None].expand(-1, -1, pairs)
    start = torch.tensor([n - t for n, t in zip(lens, new)])
    return (start[:, None] + torch.arange(S))[..., None].expand(-1, -1, pairs)


def values(pages, scale):
    """The fp64 values of a cache's pages."""
    x = pages.double() if pages.dtype != torch.float8_e4m3fn else pages.float().double()
    return x if scale is None else x * scale.double()[:, :, None, None]


def check_appended(before, after, rows, size, table, lens, new):
    """Holds one side (keys or values) of a cache after an append to the definition.

    before, after: (pages, scale or None) on the CPU; rows (B, H, S, D) fp64 as they should be cached,
    size the |a| + |b| of their rotation."""
    (p0, s0), (p1, s1) = before, after
    P, H = p0.shape[2], p0.shape[1]
    u = 2.0 ** -4 if s0 is not None else torch.finfo(p0.dtype).eps / 2
    v0, v1 = values(p0, s0), values(p1, s1)
    touched = torch.zeros(p0.shape[0], P, dtype=torch.bool)
    for b, (n, t) in enumerate(zip(lens, new)):
        start = n - t
        if t == 0:
            continue
        for j0 in range(start // P * P, n, P):
            page = int(table[b, j0 // P])
            lo, hi = max(start - j0, 0), min(n - j0, P)
            touched[page, lo:hi] = True
            x = rows[b, :, j0 + lo - start: j0 + hi - start]
            err = size[b, :, j0 + lo - start: j0 + hi - start] * 2.0 ** -20
            floor = torch.full((H, 1, 1), 2.0 ** -25 if p0.dtype == torch.float16 else 0.0, dtype=torch.float64)
            if s0 is not None:
                finite = torch.where(x.isfinite(), x.abs(), 0.0)
                for h in range(H):
                    top, slack = finite[h].max().item(), err[h].max().item()
                    allowed = {scale_for(max(top + d, 0.0)) for d in (-slack, 0.0, slack)}
                    if lo > 0:
                        allowed = {max(a, s0[page, h].item()) for a in allowed}
                    assert s1[page, h].item() in allowed, (s1[page, h].item(), allowed)
                    if lo > 0:  # the slots before, in the new scale
                        got, want = v1[page, h, :lo], code(v0[page, h, :lo] / s1[page, h].double()) * s1[page, h].double()
                        assert torch.equal(got.nan_to_num(nan=1e300), want.nan_to_num(nan=1e300))
                        touched[page, :lo] = True
                floor = s1[page].double()[:, None, None] * 2.0 ** -10
                x = x.clamp(-448.0 * s1[page].double()[:, None, None], 448.0 * s1[page].double()[:, None, None])
            got = v1[page, :, lo:hi]
            assert torch.equal(got.isnan(), x.isnan())
            bound = torch.maximum(u * x.abs(), floor) + err
            over = ((got - x).abs() - bound)[~x.isnan()]
            assert over.numel() == 0 or over.max().item() <= 0, f"{over.max().item():.3e} over its bound"
            if s0 is not None:
                touched[page, hi:] = True  # (no meaning: a new scale for the same codes)
    raw = lambda p: p.view(torch.uint8) if p.dtype == torch.float8_e4m3fn else p.view(torch.int16)  # noqa: E731
    same = (raw(p0) == raw(p1)).all(-1).all(1)
    assert bool((same | touched).all()), "slots outside the call's rows changed"
    if s0 is not None:
        untouched = ~touched.any(1)
        assert torch.equal(s0[untouched], s1[untouched])
