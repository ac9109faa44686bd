"""Appending to a paged cache and reading it back where places pass 32 bits: the buffers themselves are looked at, element
by element, not only what another call makes of them."""
import pytest
import torch

from cache_reference import check_appended, positions_of, rotate
from test_kv_cache_gpu import E4M3, make_cache, on_gpu

pytestmark = pytest.mark.gpu

LONGEST = (1 << 31) - 16


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


@pytest.mark.parametrize("eight", [False, True])
def test_places_in_a_cache_of_more_than_32_bits(eight):
    """Pages at both ends of a cache of more than 2^32 elements: rows are where they belong, every other page is as it was,
    and reading back and attention take them from there."""
    sdpa = _sdpa()
    n_pages, P, D, Hkv, n = 130, 256, 128, 1032, 300
    dtype = E4M3 if eight else torch.bfloat16
    raw = torch.zeros(2, n_pages, Hkv, P, D, dtype=torch.uint8 if eight else torch.bfloat16, device="cuda")
    assert raw[0].numel() > 1 << 32
    pages = [raw[i].view(dtype) for i in range(2)]
    cache = sdpa.KVCache(*pages, *([torch.ones(n_pages, Hkv, device="cuda") for _ in range(2)] if eight else []))
    table, lens = torch.tensor([[129, 0]], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(int(eight))
    rows = [torch.randn(1, Hkv, n, D, device="cuda", generator=g).bfloat16() for _ in range(2)]
    sdpa.kv_append(*rows, cache, table, lens)
    back = sdpa.kv_gather(cache, table, lens, n)
    sdpa.check_device_status()
    kept = []
    for side, x in enumerate(rows):
        for p in range(1, 129):
            assert not raw[side, p].view(torch.int64).any(), f"page {p} was written"
        held = torch.cat((pages[side][129], pages[side][0, :, : n - P]), 1).float()
        if eight:  # a code is off by 2^-4 of the value, or half of the smallest step, 2^-10 of its page's scale
            s = cache[2 + side]
            assert bool((s[1:129] == 1).all())
            at = torch.cat((s[129, :, None].expand(-1, P), s[0, :, None].expand(-1, n - P)), 1)[..., None]
            held = held * at
            assert bool(((held - x[0].float()).abs() <= torch.maximum(2.0 ** -4 * x[0].float().abs(), 2.0 ** -10 * at)).all())
        else:
            assert torch.equal(held, x[0].float())
        assert not raw[side, 0, :, n - P:].view(torch.int64).any()
        assert torch.equal(back[side][0].float(), held)  # (codes times a power of two are bf16 numbers)
        kept.append(held)
    q = torch.randn(1, Hkv, 1, D, device="cuda", generator=g).bfloat16()
    o, _ = sdpa.sdpa_fwd_cached(q, cache, table, lens)
    sdpa.check_device_status()
    k, v = (x.double() for x in kept)
    p = torch.softmax((q[0].double() @ k.mT) / D ** 0.5, -1)
    want, spread = (p @ v), (p @ v.abs())
    # One rounding of O, one of each weight (fp16 over codes), and 2^-15 of what is summed for scores and sums.
    u, u_p = 2.0 ** -8, 2.0 ** -11 if eight else 2.0 ** -8
    assert bool(((o[0].double() - want).abs() <= u * want.abs() + (u_p + 2.0 ** -15) * spread * (1 + u)).all())


@pytest.mark.parametrize("eight", [False, True])
def test_appending_at_the_end_of_the_longest_table(eight):
    """The last 37 positions of a table of 2^31 - 16, rotated there."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(3)
    P, D, H, S = 16, 32, 2, 37
    dtype = E4M3 if eight else torch.bfloat16
    before = make_cache(g, 9, H, P, D, dtype)
    table = torch.zeros(1, LONGEST // P, dtype=torch.int32)
    table[0, -3:] = torch.tensor([5, 2, 7], dtype=torch.int32)
    cache, freq = on_gpu(before), sdpa.rope_inv_freq(D)
    k, v = (torch.randn(1, H, S, D, generator=g).bfloat16() for _ in range(2))
    sdpa.kv_append(k.cuda(), v.cuda(), cache, table.cuda(), torch.tensor([LONGEST], dtype=torch.int32).cuda(), inv_freq=freq)
    sdpa.check_device_status()
    after = [None if t is None else t.cpu() for t in cache]
    rows, size = rotate(k, freq.cpu(), positions_of([LONGEST], [S], S, D // 2))
    check_appended((before[0], before[2]), (after[0], after[2]), rows, size, table, [LONGEST], [S])
    rows, size = rotate(v, None, None)
    check_appended((before[1], before[3]), (after[1], after[3]), rows, size, table, [LONGEST], [S])


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
