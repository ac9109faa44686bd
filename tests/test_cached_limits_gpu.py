"""Attention over a paged cache at the longest table that it takes, 2^31 - 16 positions, in pages of 16: the table
names a few pages over and over, so that the cache itself is small."""
import math

import pytest
import torch

from test_cached_attention_gpu import check, reference
from test_kv_cache_gpu import E4M3, make_cache, on_gpu

pytestmark = pytest.mark.gpu

LONGEST = (1 << 31) - 16


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


@pytest.mark.parametrize("io,eight", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True), (torch.float16, True)])
@pytest.mark.parametrize("Sq,slope", [(1, 0.0), (5, 0.0), (5, 0.05), (40, 0.0), (40, 0.05)])
def test_window_at_the_end_of_the_longest_table(io, eight, Sq, slope):
    """A sequence that fills the table, beside a short one: what its rows see are its first 5 pages and its last 20, so
    the answer is that of these 25 pages alone. The page that all other entries name is NaN."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(Sq)
    P, D, W, F = 16, 32, 200, 0 if slope else 70  # (the first keys' distances would not be those of the 25 pages)
    cache = make_cache(g, 50, 1, P, D, E4M3 if eight else io)
    for pages in cache[:2]:
        pages.view(torch.uint8 if eight else torch.int16)[0] = 0x7F if eight else 0x7FFF
    seen = torch.stack([torch.arange(1, 26), torch.arange(26, 26 + 25) % 50]).to(torch.int32)
    table = torch.zeros(2, LONGEST // P, dtype=torch.int32, device="cuda")
    table[0, :5], table[0, -20:] = seen[0, :5].cuda(), seen[0, 5:].cuda()
    table[1, :19] = seen[1, :19].cuda()
    q = torch.randn(2, 2, Sq, D, generator=g).to(io)
    slopes = torch.full((2,), slope) if slope else None
    got = sdpa.sdpa_fwd_cached(q.cuda(), on_gpu(cache), table, torch.tensor([LONGEST, 300], dtype=torch.int32).cuda(),
                               window_left=W, first_keys=F, alibi_slopes=None if slopes is None else slopes.cuda())
    sdpa.check_device_status()
    check(got, reference(q, cache, seen, [400, 300], [Sq] * 2, window=W, first=F, slopes=slopes))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("Sq", [1, 40])
def test_all_of_the_longest_table(eight, Sq):
    """Queries of zeros see every key alike: O is the mean of the values, which are 1, and the LSE log n. Sums of a
    thread are whole multiples of one weight below 2^24 of them, exact in fp32; at most 2,000 parts are joined, each
    with one rounding of 2^-24, and so are 8 threads of a row before them."""
    sdpa = _sdpa()
    P, D = 16, 16
    dtype = E4M3 if eight else torch.bfloat16
    cache = sdpa.kv_cache(2, 1, P, D, dtype=dtype)
    cache.v.copy_(torch.ones(2, 1, P, D))
    table = torch.zeros(1, LONGEST // P, dtype=torch.int32, device="cuda")
    table[0, ::2] = 1
    q = torch.zeros(1, 1, Sq, D, dtype=torch.bfloat16, device="cuda")
    o, lse = sdpa.sdpa_fwd_cached(q, cache, table, torch.tensor([LONGEST], dtype=torch.int32).cuda(), causal=False)
    sdpa.check_device_status()
    assert (o.float() - 1).abs().max().item() <= 2.0 ** -8
    assert (lse.double() - math.log(LONGEST)).abs().max().item() <= 2010 * 2.0 ** -24 + 2.0 ** -18
