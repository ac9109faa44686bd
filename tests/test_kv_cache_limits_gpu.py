"""Appending to a paged cache and reading it back where places pass 32 bits: the buffers themselves are looked at, element
by element, not only what another call makes of them."""
import pytest
import torch

from test_kv_cache_gpu import make_cache, on_gpu

pytestmark = pytest.mark.gpu

LONGEST = (1 << 31) - 16


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def test_reading_the_longest_table_back():
    """All positions of a table of 2^31 - 16, 64 GB a side, zeros past the length."""
    sdpa = _sdpa()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 170 << 30:
        pytest.skip("takes 140 GB of free device memory")
    P, D, n = 16, 16, LONGEST - 40
    cache = on_gpu(make_cache(torch.Generator().manual_seed(4), 4, 1, P, D, torch.bfloat16))
    table = torch.zeros(1, LONGEST // P, dtype=torch.int32, device="cuda")
    table[0, 1::2] = 3
    out = sdpa.kv_gather(cache, table, torch.tensor([n], dtype=torch.int32).cuda())
    sdpa.check_device_status()
    for side in range(2):
        pair = torch.cat((cache[side][0, 0], cache[side][3, 0])).view(torch.int16)  # 32 positions
        x = out[side].view(torch.int16).view(-1, D)
        for at in range(0, n // 32 * 32, 1 << 25):
            some = x[at: min(at + (1 << 25), n // 32 * 32)].view(-1, 32, D)
            assert bool((some == pair).all()), f"positions from {at}"
        assert torch.equal(x[n // 32 * 32: n], pair[: n % 32]) and not x[n:].any()
    del out, x, some
    torch.cuda.empty_cache()
