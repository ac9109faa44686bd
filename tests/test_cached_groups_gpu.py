"""Attention over a paged cache where 9 to 16 rows a key/value head (and 17 to 32 of up to 64 columns) share a tile of the
few-rows kernel, at head dims up to 128 and with modified scores; and weights far below a row's largest. Against the 64-bit
reference, with the bounds of test_cached_attention_gpu.py."""
import math

import pytest
import torch

from test_cached_attention_gpu import TYPES, case, check, reference
from test_kv_cache_gpu import E4M3, on_gpu

pytestmark = pytest.mark.gpu


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(9, 1), (12, 1), (30, 2), (48, 3)])
@pytest.mark.parametrize("D", [80, 128])
def test_many_heads_to_one(io, eight, Hq, Hkv, D):
    case(io, eight, [400, 33, 1], 1, Hq, Hkv, 32, D, seed=Hq)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq,group", [(2, 5), (4, 4), (5, 3), (16, 1)])
@pytest.mark.parametrize("D", [80, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_a_few_queries_of_some_heads(io, eight, Sq, group, D, causal):
    case(io, eight, [Sq, Sq + 1, 500, 333], Sq, 2 * group, 2, 16, D, seed=Sq, causal=causal)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("window,first", [(0, 1), (64, 16), (300, 37)])
def test_windows(io, eight, window, first):
    case(io, eight, [6, 250, 1111], 6, 4, 2, 64, 128, seed=window, window=window, first=first)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq,D", [(1, 64), (4, 64), (4, 80), (5, 128), (6, 64), (10, 64), (50, 64), (50, 80)])
@pytest.mark.parametrize("kw", [{"softcap": 20.0}, {"slopes": True}, {"softcap": 5.0, "slopes": True, "sink": True, "window": 50, "first": 3}])
def test_modified_scores(io, eight, Sq, D, kw):
    """3 rows a head, 12 and 15, 18 and 30, and 150."""
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = 2.0 ** (-torch.arange(1, 7).float())
    if "sink" in kw:
        kw["sink"] = torch.randn(6, generator=torch.Generator().manual_seed(Sq)) * 3
    case(io, eight, [Sq, 200, 777], Sq, 6, 2, 16, D, seed=Sq + D, **kw)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq", [1, 6, 12, 40, 140])
def test_weights_far_below_the_largest(io, eight, Sq):
    """One key in 64 has e^18 times the weight of every other one, and zeros for a value: O is what the others leave, weights
    of 2^-26 of the largest."""
    n, P, D = 1000, 16, 64
    k, v = torch.zeros(63, 1, P, D), torch.zeros(63, 1, P, D)
    k[::4, :, 0, 0] = 4.0
    v[:] = 1024.0 * 2.0 ** -torch.randint(0, 3, v.shape, generator=torch.Generator().manual_seed(Sq))
    v[::4, :, 0] = 0.0
    scales = [torch.full((63, 1), 4.0) for _ in range(2)]
    cache = ((k / 4).to(E4M3), (v / 4).to(E4M3), *scales) if eight else (k.to(io), v.to(io), None, None)
    q = torch.zeros(1, 2, Sq, D, dtype=io)
    q[..., 0] = 4.5
    table = torch.arange(63, dtype=torch.int32)[None]
    got = _sdpa().sdpa_fwd_cached(q.cuda(), on_gpu(cache), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                  scale=1.0, causal=False)
    want = reference(q, cache, table, [n], [Sq], scale=1.0, causal=False)
    assert (want[2] < want[0].abs() / 8).all() and (want[0].abs() / 1024 < 64 * math.exp(-18)).all()
    check(got, want)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Sq,Hq,D", [(1, 2, 64), (1, 8, 128), (3, 8, 128), (4, 8, 64), (8, 8, 64), (5, 8, 48)])
@pytest.mark.parametrize("n", [9, 40, 700])
def test_weights_are_not_rounded_to_the_cache_s_type(io, Sq, Hq, D, n):
    """Few rows over 16-bit pages: a weight counts as a rounded one and the rest of it, rounded too, off by u^2 of itself and
    not by u, so that O is held to its own rounding where positive and negative values all but cancel. (Below fp16's
    normal numbers what is left out is in the bound's term of small weights.)"""
    g = torch.Generator().manual_seed(Sq + n)
    P = 16
    k, v = (torch.randn(-(-n // P), 2, P, D, generator=g).to(io) for _ in range(2))
    q = torch.randn(1, Hq, Sq, D, generator=g).to(io)
    table = torch.arange(-(-n // P), dtype=torch.int32)[None]
    got = _sdpa().sdpa_fwd_cached(q.cuda(), on_gpu((k, v, None, None)), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    o, lse, bo, bl = reference(q, (k, v, None, None), table, [n], [Sq])
    size = reference(q, (k, v.abs(), None, None), table, [n], [Sq])[0]  # P |V|
    u = 2.0 ** -8 if io == torch.bfloat16 else 2.0 ** -11
    check(got, (o, lse, bo - (u - u * u) * size, bl))


@pytest.mark.parametrize("io,eight", [(torch.bfloat16, False), (torch.float16, True)])
@pytest.mark.parametrize("B,Sq", [(300, 1), (140, 6), (700, 17)])
def test_more_sequences_than_a_block_has_threads(io, eight, B, Sq):
    """Several entries a thread of the schedule (128 threads, or 640 of the many-rows kernel), a third of them without a key."""
    g = torch.Generator().manual_seed(B)
    lens = [int(n) * int(z) for n, z in zip(torch.randint(Sq, 90, (B,), generator=g), torch.randint(0, 3, (B,), generator=g) > 0)]
    new = [min(Sq, n) for n in lens]
    case(io, eight, lens, Sq, 2, 1, 16, 64, new=new, seed=B, window=40, first=2)


@pytest.mark.parametrize("eight", [False, True])
def test_more_row_tiles_than_a_block_has_threads(eight):
    """One chunk of 83,000 rows a head in 649 tiles, behind a prefix; a few rows of it are checked by calls of their own."""
    sdpa = _sdpa()
    g = torch.Generator(device="cuda").manual_seed(1)
    S, P, D = 83_000, 256, 16
    n = S + 100
    cache = sdpa.kv_cache(-(-n // P), 1, P, D, dtype=E4M3 if eight else torch.bfloat16)
    table = torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    k, v, q = (torch.randn(1, 1, m, D, device="cuda", generator=g).bfloat16() for m in (n, n, S))
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    sdpa.kv_append(k, v, cache, table, lens)
    o, lse = sdpa.sdpa_fwd_cached(q, cache, table, lens, window_left=500, first_keys=3)
    sdpa.check_device_status()
    held = type(cache)(*(None if t is None else t.cpu() for t in cache))
    for i in (0, 1, 127, 128, 41_111, S - 130, S - 1):
        want = reference(q[:, :, i: i + 1].cpu(), held, table.cpu(), [n - S + i + 1], [1], window=500, first=3)
        check((o[:, :, i: i + 1], lse[:, :, i: i + 1]), want)
