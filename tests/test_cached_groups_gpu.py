"""Attention over a paged cache with weights far below a row's largest. Against the 64-bit reference, with the bounds of
test_cached_attention_gpu.py."""
import math

import pytest
import torch

from test_cached_attention_gpu import TYPES, check, reference
from test_kv_cache_gpu import E4M3, on_gpu

pytestmark = pytest.mark.gpu


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


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
