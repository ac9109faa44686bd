"""Appending to a paged cache and reading it back, on the GPU, against the 64-bit reference
(bounds in cache_reference.py)."""
import pytest
import torch

from cache_reference import check_appended, code, positions_of, rotate, values

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def make_cache(g, n_pages, Hkv, P, D, dtype, spread=0):
    """A cache of random pages (CPU): values around 1, in 8 bits with scales 2^-10 .. 2^-6, wider by `spread`."""
    x = torch.randn(2, n_pages, Hkv, P, D, generator=g)
    if dtype != E4M3:
        k, v = (x * 1.0).to(dtype)
        return k, v, None, None
    e = torch.randint(-10 - spread, -6 + spread, (2, n_pages, Hkv), generator=g)
    codes = (x * 60).clamp(-448, 448).to(E4M3)
    return codes[0], codes[1], (2.0 ** e[0]).float(), (2.0 ** e[1]).float()


def on_gpu(cache):
    return _sdpa().KVCache(*(None if t is None else t.cuda() for t in cache))


def table_for(g, B, per_row, n_pages):
    return torch.randperm(n_pages, generator=g)[: B * per_row].view(B, per_row).to(torch.int32)


def append_case(dtype, io, lens, new, S, Hq, Hkv, P, D, rot, seed=0, interleaved=False, mult=1.0, axes=None,
                positions=None, gain=1.0, spread=0, layout="bshd"):
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(seed)
    B, per_row = len(lens), max(1, -(-max(lens) // P))
    n_pages = B * per_row + 3
    before = make_cache(g, n_pages, Hkv, P, D, dtype, spread)
    table = table_for(g, B, per_row, n_pages)
    cache = on_gpu(before)
    rows = [(torch.randn(B, S, H, D, generator=g) * gain).to(io) for H in (Hq, Hkv, Hkv)]
    if layout == "bshd":
        q, k, v = (r.cuda().transpose(1, 2) for r in rows)
    elif layout == "odd":  # rows that no 16-byte access can take
        q, k, v = (torch.zeros(B, S, r.shape[2], D + 3, dtype=io).cuda()[..., 1:D + 1].copy_(r).transpose(1, 2) for r in rows)
    else:
        q, k, v = (r.transpose(1, 2).contiguous().cuda() for r in rows)
    freq = None if rot == 0 else sdpa.rope_inv_freq(rot)
    out = sdpa.kv_append(k, v, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                         seq_q_lens=None if all(n == S for n in new) else torch.tensor(new, dtype=torch.int32).cuda(),
                         q=q if Hq else None, inv_freq=freq, mult=mult, interleaved=interleaved,
                         positions=None if positions is None else positions.cuda(),
                         axes=None if axes is None else axes.cuda())
    sdpa.check_device_status()
    f = None if freq is None else freq.cpu()
    pos = positions_of(lens, new, S, rot // 2, positions, axes)
    rows = [r.transpose(1, 2) for r in rows]
    after = [None if t is None else t.cpu() for t in cache]
    k_rows, k_size = rotate(rows[1], f, pos, mult, interleaved)
    check_appended((before[0], before[2]), (after[0], after[2]), k_rows, k_size, table, lens, new)
    v_rows, v_size = rotate(rows[2], None, None)
    check_appended((before[1], before[3]), (after[1], after[3]), v_rows, v_size, table, lens, new)
    if Hq:
        assert out.is_contiguous()
        y, size = rotate(rows[0], f, pos, mult, interleaved)
        u = torch.finfo(io).eps / 2
        bound = u * y.abs() + size * 2.0 ** -20 + (2.0 ** -25 if io == torch.float16 else 0.0)
        fits = y.abs() < 3e38  # (rows with infinities, or beyond fp32: the outputs are none of numbers)
        assert ((out.cpu().double() - y).abs() - bound)[fits].max().item() <= 0
        assert torch.equal(out.cpu().isnan(), y.isnan())
    return cache, table, after


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_page_sizes(io, eight, P):
    """Rows that begin and end inside pages, at their borders, and one to a page."""
    lens = [1, 16, P, P + 1, 3 * P - 1, 300]
    new = [min(n, t) for n, t in zip(lens, [1, 16, 7, 37, 37, 1])]
    append_case(E4M3 if eight else io, io, lens, new, 37, 4, 2, P, 64, 64, seed=P)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (80, 80), (96, 48), (112, 20), (16, 16), (48, 6), (64, 0)])
@pytest.mark.parametrize("layout", ["bshd", "bhsd", "odd"])
def test_columns_and_layouts(eight, D, rot, layout):
    io = torch.bfloat16
    append_case(E4M3 if eight else io, io, [50, 23], [19, 19], 19, 3, 3, 16, D, rot, seed=D + rot, layout=layout,
                interleaved=rot % 4 == 0 and rot != 64, mult=1.25)


@pytest.mark.parametrize("B,S,Hq,Hkv", [(1, 1, 1, 1), (64, 1, 32, 8), (1, 4000, 2, 1), (3, 5, 0, 2), (2, 129, 41, 1)])
@pytest.mark.parametrize("eight", [False, True])
def test_sizes_and_heads(B, S, Hq, Hkv, eight):
    lens = [S + 37 * b for b in range(B)]
    append_case(E4M3 if eight else torch.bfloat16, torch.bfloat16, lens, [S] * B, S, Hq, Hkv, 16, 128, 128, seed=S)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("shape", ["(S,)", "(B, S)", "axes (n, S)", "axes (n, B, S)"])
def test_given_positions(eight, shape):
    g = torch.Generator().manual_seed(4)
    B, S = 2, 21
    dims = {"(S,)": (S,), "(B, S)": (B, S), "axes (n, S)": (3, S), "axes (n, B, S)": (3, B, S)}[shape]
    positions = torch.randint(-50, 100000, dims, generator=g, dtype=torch.int32)
    axes = torch.tensor([0] * 8 + [1, 2] * 12, dtype=torch.int32) if "axes" in shape else None
    append_case(E4M3 if eight else torch.float16, torch.float16, [40, 21], [S, S], S, 4, 2, 32, 64, 64,
                positions=positions, axes=axes)


@pytest.mark.parametrize("gain", [1e-30, 1e-12, 2.0 ** -40, 1.0, 100.0, 1e10, 1e38])
def test_scales_of_small_and_large_values(gain):
    """Scales grow and stay, older slots are rounded anew, far apart scales meet in a page."""
    append_case(E4M3, torch.bfloat16, [40, 100, 33], [20, 20, 1], 20, 2, 2, 64, 64, 32, gain=gain, spread=8)


def test_values_that_no_scale_counts():
    """Infinities saturate, NaN stay; zeros alone give the smallest scale."""
    sdpa = _sdpa()
    cache = sdpa.kv_cache(3, 1, 16, 16, E4M3)
    k = torch.ones(1, 1, 16, 16).bfloat16()
    k[0, 0, 0, 0], k[0, 0, 1, 1], k[0, 0, 2, 2] = float("inf"), float("nan"), -float("inf")
    v = torch.zeros(1, 1, 16, 16).bfloat16()
    sdpa.kv_append(k.cuda(), v.cuda(), cache, torch.tensor([[2]], dtype=torch.int32).cuda(),
                   torch.tensor([16], dtype=torch.int32).cuda())
    got = values(cache.k.cpu(), cache.k_scale.cpu())[2, 0]
    assert cache.k_scale[2, 0].item() == 2.0 ** -8 and cache.v_scale[2, 0].item() == 2.0 ** -64
    assert got[0, 0] == 448 * 2.0 ** -8 and got[2, 2] == -448 * 2.0 ** -8 and got[1, 1].isnan()
    got[0, 0] = got[2, 2] = got[1, 1] = 1.0
    assert bool((got == 1.0).all()) and not cache.v.float().any()
    sdpa.check_device_status()


@pytest.mark.parametrize("eight", [False, True])
def test_token_by_token_as_at_once(eight):
    """A sequence appended in pieces holds the same rows in 16 bits, and in 8 bits rows within the
    bounds of each step (the last step's check covers all that the page's scale changed)."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(9)
    n, P, D = 75, 16, 64
    k, v = (torch.randn(1, 2, n, D, generator=g).bfloat16().cuda() for _ in range(2))
    freq = sdpa.rope_inv_freq(D)
    table = torch.tensor([[4, 1, 0, 3, 5]], dtype=torch.int32).cuda()
    caches = [sdpa.kv_cache(6, 2, P, D, E4M3 if eight else torch.bfloat16) for _ in range(2)]
    at = 0
    for step in (1, 1, 1, 20, 5, 1, 30, 16):
        lens = torch.tensor([at + step], dtype=torch.int32).cuda()
        sdpa.kv_append(k[:, :, at:at + step], v[:, :, at:at + step], caches[0], table, lens, inv_freq=freq)
        at += step
    sdpa.kv_append(k, v, caches[1], table, torch.tensor([n], dtype=torch.int32).cuda(), inv_freq=freq)
    a, b = (sdpa.kv_gather(c, table, torch.tensor([n], dtype=torch.int32).cuda()) for c in caches)
    for x, y in zip(a, b):
        if not eight:
            assert torch.equal(x, y)
            continue
        # The scales agree (the largest value decides in any order), and a value that went through a
        # smaller scale first was rounded there only below 2^-6 of it: half a step twice.
        step = torch.cat([s[table[0].long()] for s in (caches[0].k_scale if x is a[0] else caches[0].v_scale,)])
        unit = step.repeat_interleave(P, 0)[:n].T[None, :, :, None].double()
        assert ((x[:, :, :n].double() - y[:, :, :n].double()).abs() <= unit * 2.0 ** -9).all()
    if eight:
        assert torch.equal(caches[0].k_scale[table[0].long()], caches[1].k_scale[table[0].long()])
        assert torch.equal(caches[0].v_scale[table[0].long()], caches[1].v_scale[table[0].long()])


def test_rows_written_again():
    """Positions appended once more (a proposal taken back) hold the new rows; a page whose first slot
    is among them starts anew, its scale included."""
    cache, table, _ = append_case(E4M3, torch.bfloat16, [40], [40], 40, 0, 2, 16, 64, 0, gain=50.0)
    sdpa = _sdpa()
    before = [t.cpu() for t in cache]
    rows = torch.randn(1, 2, 12, 64).bfloat16()
    sdpa.kv_append(rows.cuda(), rows.cuda(), cache, table.cuda(), torch.tensor([36], dtype=torch.int32).cuda())
    after = [t.cpu() for t in cache]
    check_appended((before[0], before[2]), (after[0], after[2]), rows.double(), rows.double() * 0, table, [36], [12])
    assert after[2][table[0, 2].long()].max() < before[2][table[0, 2].long()].min()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("S", [1, 17, 96, None])
def test_gather(eight, io, S):
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(3)
    cache = make_cache(g, 23, 3, 32, 80, E4M3 if eight else io)
    table = table_for(g, 4, 5, 23)
    lens = [0, 1, 95, 160]
    k, v = sdpa.kv_gather(on_gpu(cache), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), S, dtype=io)
    n = 160 if S is None else S
    assert k.shape == v.shape == (4, 3, n, 80)
    for got, pages, scale in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        want = values(pages, scale)[table.long()].transpose(1, 2).flatten(2, 3)[:, :, :n].to(io)
        for b, m in enumerate(lens):
            want[b, :, m:] = 0
        assert torch.equal(got.cpu(), want)
    sdpa.check_device_status()


def test_pages_and_lengths_outside_the_cache_are_skipped_and_reported():
    """Bad page ids and lengths past the table: nothing is written for them, the rest is, and the
    status says so once. (Every access is checked against the buffers before it is made.)"""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(5)
    for dtype in (E4M3, torch.bfloat16):
        for table, lens in (([[0, 7, 2]], 40), ([[0, -1, 2]], 40), ([[0, 1, 2]], 60), ([[0, 1, 2]], -3), ([[1 << 30, 1, 2]], 40)):
            before = make_cache(g, 4, 2, 16, 32, dtype)
            cache = on_gpu(before)
            rows = torch.randn(1, 2, 40, 32, generator=g).bfloat16().cuda()
            t, n = torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor([lens], dtype=torch.int32).cuda()
            sdpa.kv_append(rows, rows, cache, t, n)
            with pytest.raises(sdpa.SdpaError, match="SDPA_ERR_PAGE"):
                sdpa.check_device_status()
            sdpa.check_device_status()
            assert torch.equal(cache.k[3].view(torch.uint8).cpu(), before[0][3].view(torch.uint8))
            k, v = sdpa.kv_gather(cache, t, n)
            with pytest.raises(sdpa.SdpaError, match="SDPA_ERR_PAGE"):
                sdpa.check_device_status()
            for j, page in enumerate(table[0]):
                if not 0 <= page < 4:
                    assert not k[:, :, 16 * j: 16 * j + 16].any() and not v[:, :, 16 * j: 16 * j + 16].any()


@pytest.mark.parametrize("eight", [False, True])
def test_captured_and_replayed(eight):
    """One graph appends a token a replay, its lengths and rows updated in place."""
    sdpa = _sdpa()
    B, Hkv, P, D = 3, 2, 16, 64
    cache, ref = (sdpa.kv_cache(20, Hkv, P, D, E4M3 if eight else torch.bfloat16) for _ in range(2))
    table = torch.randperm(20)[:15].view(3, 5).to(torch.int32).cuda()
    lens = torch.tensor([0, 15, 40], dtype=torch.int32).cuda()
    k, v, q = (torch.zeros(B, H, 1, D).bfloat16().cuda() for H in (Hkv, Hkv, 4))
    q_out = torch.empty_like(q)
    freq = sdpa.rope_inv_freq(D)
    call = lambda c: sdpa.kv_append(k, v, c, table, lens, q=q, inv_freq=freq, q_out=q_out)  # noqa: E731
    lens += 1  # (an empty sequence has no last row to append)
    call(sdpa.kv_cache(20, Hkv, P, D, E4M3 if eight else torch.bfloat16))
    lens -= 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache)
    for _ in range(5):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape))
        lens += 1
        graph.replay()
        captured = q_out.clone()
        call(ref)
        assert torch.equal(captured, q_out)
    for a, b in zip(cache, ref):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    sdpa.check_device_status()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("P,D,rot,interleaved,mult", [(32, 128, 128, False, 1.0), (64, 128, 64, True, 1.25), (256, 64, 64, False, 1.0),
                                                      (16, 80, 40, True, 1.0), (16, 16, 2, False, 0.8)])
def test_codes_of_the_exact_rotation(io, P, D, rot, interleaved, mult):
    """Codes are those of the rotation in 64 bits: a value as near to a tie as 2^-31 (|a| + |b|) may fall on either side
    of it (sine and cosine are off by 2^-33 each, their products and sum by 2^-46), any other on its own."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(P + rot)
    B, S, Hkv = 2, 700, 3
    per_row = -(-S // P)
    cache = sdpa.kv_cache(B * per_row, Hkv, P, D, dtype=E4M3)
    table = table_for(g, B, per_row, B * per_row)
    k = torch.randn(B, Hkv, S, D, generator=g).to(io)
    freq, where = sdpa.rope_inv_freq(rot), torch.randint(-50, 100000, (B, S), generator=g, dtype=torch.int32)
    sdpa.kv_append(k.cuda(), k.cuda(), cache, table.cuda(), torch.tensor([S, S], dtype=torch.int32).cuda(), inv_freq=freq,
                   mult=mult, interleaved=interleaved, positions=where.cuda())
    x, size = rotate(k, freq.cpu(), positions_of([S] * B, [S] * B, S, rot // 2, where), float(torch.tensor(mult)), interleaved)
    codes, scale = cache.k.float().double().cpu(), cache.k_scale.double().cpu()
    differ = 0
    for b in range(B):
        pages = table[b].long()
        got = codes[pages].transpose(0, 1).flatten(1, 2)[:, :S]
        s = scale[pages].T.repeat_interleave(P, 1)[:, :S, None]
        # (At position 0 nothing turns and a 16th of the 8-bit values are ties to 4 bits: exact, so no allowance.)
        d = size[b] * 2.0 ** -31 * (where[b] != 0)[None, :, None]
        low, high = code((x[b] - d) / s), code((x[b] + d) / s)
        assert bool(((got == low) | (got == high)).all())
        differ += (low != high).sum().item()
    assert differ <= 2  # (of 10^5 values, each 2^-26 of its step from a tie or nearer: one in 10^7)
