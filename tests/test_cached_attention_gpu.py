"""Attention over a paged cache on the GPU against 64-bit attention over the values that the
cache holds.

Bounds, elementwise; P the exact weights, u half a step of the io type, A = P |V|:
  |O_gpu - O| <= u |O| [rounded once] + u_P A [weights rounded to the type that they meet values in: the cache's,
                 bf16 2^-8 or fp16 2^-11; over codes fp16, to which these are widened]
                 + 2 e A [scores, in the numerator and the sum] + w 2^-31 sum |V| [weights below fp16's
                 smallest step: taken times 2^6 of a reference at most the row's largest, half a step 2^-25]
                 (fp16 results below 2^-14: 2^-25 more; bf16 below 2^-126, where its step is 2^-133: 2^-134;
                 beside a sink that far above, weights below fp32's normal numbers are 0: 2^-126 |v|max more)
  |LSE_gpu - LSE| <= e + 2^-19
  e = g (D + 16) max sum |q k| scale + g (|x|max + |LSE| + 8) + g slope distance + n 2^-24 + 2^-20
      g = 2^-23; n keys a row in the sum; 2^-20: exponentials and logarithms of a few units, in a chain of three
  (8 bits with bf16 queries: they are fp16 times a power of two, off by 2^-39 of the row's largest; in A and
  the last term V counts with its scale, and w is the largest P times value scale.)"""
import math

import pytest
import torch

from cache_reference import values
from test_kv_cache_gpu import E4M3, make_cache, on_gpu, table_for

pytestmark = pytest.mark.gpu
G = 2.0 ** -23


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def reference(q, cache, table, lens, new, *, causal=True, window=-1, first=0, sink=None, softcap=0.0, slopes=None, scale=None):
    """(O, LSE, bound of O, bound of LSE) in fp64, on the GPU's fp64 units."""
    k_pages, v_pages, ks, vs = (None if t is None else t.cuda() for t in cache)
    B, Hq, Sq, D = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    rep, dev = Hq // Hkv, "cuda"
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    io = q.dtype
    u, u_p = torch.finfo(io).eps / 2, 2.0 ** -11 if io == torch.float16 or ks is not None else 2.0 ** -8
    o = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device=dev)
    bo, bl = torch.full_like(o, 2.0 ** -149), torch.full_like(lse, 2.0 ** -19)
    if sink is not None:
        lse[:] = sink.double().cuda()[None, :, None]
        bl[:] += lse.abs().nan_to_num(posinf=0.0) * G
    for b, (n, t) in enumerate(zip(lens, new)):
        if n == 0 or t == 0:
            continue
        at = table[b, : -(-n // P)].long().cuda()
        take = lambda pages, s: values(pages[at], None if s is None else s[at]).transpose(0, 1).flatten(1, 2)[:, :n]  # noqa: E731
        K, V = take(k_pages, ks), take(v_pages, vs)  # (Hkv, n, D)
        vscale = torch.ones(Hkv, n, dtype=torch.float64, device=dev) if vs is None else \
            vs[at].double().T.repeat_interleave(P, 1)[:, :n]
        j, place = torch.arange(n, device=dev)[None], (n - t + torch.arange(t, device=dev))[:, None]
        see = (j <= place) if causal else (j < n).expand(t, n)
        if window >= 0:
            see = see & ((j >= place - window) | (j < first))
        see = see & (torch.arange(t, device=dev)[:, None] >= 0)
        for h in range(Hq):
            qh, kh, vh = q[b, h, :t].double().cuda(), K[h // rep], V[h // rep]
            y = qh @ kh.T * scale
            size = (qh.abs() @ kh.abs().T * scale).masked_fill(~see, 0.0)
            x = softcap * torch.tanh(y / softcap) if softcap else y
            dist = (place - j).abs().double()
            sl = 0.0 if slopes is None else slopes[h].item()
            x = torch.where(see, x - sl * dist, -math.inf)
            full = x if sink is None else torch.cat((x, sink[h].double().cuda().expand(t, 1)), 1)
            L = torch.logsumexp(full, 1)
            p = torch.exp(x - torch.where(L == -math.inf, 0.0, L)[:, None])
            fin = torch.where(see, x.abs(), 0.0)
            e = G * (D + 16) * size.amax(1) + G * (fin.amax(1) + torch.where(L.isfinite(), L.abs(), 0.0) + 8.0) \
                + G * abs(sl) * torch.where(see, dist, 0.0).amax(1) + see.sum(1) * 2.0 ** -24 + 2.0 ** -20
            A, out = p @ vh.abs(), p @ vh
            w = (p * vscale[h // rep]).amax(1)
            small = w[:, None] * (see.double() @ (vh.abs() / vscale[h // rep][:, None])) * 2.0 ** -31
            o[b, h, :t], lse[b, h, :t] = out, L
            bo[b, h, :t] += u * out.abs() + (u_p + 2 * e[:, None]) * A + small + (2.0 ** -25 if io == torch.float16 else 2.0 ** -134) \
                + 2.0 ** -126 * vh.abs().max()
            bl[b, h, :t] = e + 2.0 ** -19
    return o, lse, bo, bl


def check(got, want):
    o, lse = got
    eo, el, bo, bl = want
    none = el == -math.inf
    assert torch.equal(lse == -math.inf, none)
    assert not o[none].any()
    over = ((o.double() - eo).abs() - bo).max().item()
    assert over <= 0, f"O {over:.3e} over its bound"
    over = ((lse.double() - el).abs() - bl)[~none]
    assert over.numel() == 0 or over.max().item() <= 0, f"LSE {over.max().item():.3e} over its bound"


def case(io, eight, lens, Sq, Hq, Hkv, P, D, new=None, seed=0, gain=2.0, spread=0, poison=True, **kw):
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per_row = max(1, -(-max(lens) // P))
    n_pages = B * per_row + 3
    cache = make_cache(g, n_pages, Hkv, P, D, E4M3 if eight else io, spread)
    table = table_for(g, B, per_row, n_pages)
    new = [Sq] * B if new is None else new
    if poison:  # what lies behind the sequences, and in pages that none has, is NaN
        bad = torch.ones(n_pages, P, dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(-(-n // P)):
                bad[table[b, p].long(), : min(P, n - p * P)] = False
            table[b, -(-n // P):] = -1 if b % 2 else 1 << 30  # entries that no position uses
        for pages in cache[:2]:
            raw = pages.view(torch.uint8 if eight else torch.int16)
            raw.transpose(1, 2)[bad] = 0x7F if eight else (0x7FC0 if io == torch.bfloat16 else 0x7E00)
    q = (torch.randn(B, Hq, Sq, D, generator=g) * gain).to(io)
    names = {"window": "window_left", "first": "first_keys", "slopes": "alibi_slopes"}
    call = {names.get(k, k): v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    got = sdpa.sdpa_fwd_cached(q.cuda(), on_gpu(cache), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               seq_q_lens=None if new == [Sq] * B else torch.tensor(new, dtype=torch.int32).cuda(), **call)
    sdpa.check_device_status()
    check(got, reference(q, cache, table, lens, new, **kw))
    return got


TYPES = [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True), (torch.float16, True)]


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens(io, eight, P, D):
    """Lengths of one, around pages and units, and long ones; sequences without a key among them."""
    case(io, eight, [1, 0, 15, 16, 17, 63, 64, 65, 127, 129, 700, 2500], 1, 8, 2, P, D, seed=P + D)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("D", [16, 32, 48, 80, 96, 112])
def test_head_dims(io, eight, D):
    case(io, eight, [300, 77], 1, 6, 3, 32, D, seed=D)
    case(io, eight, [300, 177], 40, 6, 3, 32, D, seed=D)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 7), (5, 1), (16, 1), (17, 1), (32, 2), (33, 1), (40, 1), (64, 8), (71, 1), (128, 1)])
def test_head_groups(io, eight, Hq, Hkv):
    case(io, eight, [400, 33], 1, Hq, Hkv, 16, 64, seed=Hq)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq,group", [(2, 4), (3, 5), (5, 4), (16, 1), (17, 1), (8, 4), (33, 1), (9, 8), (130, 1), (61, 3), (300, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_queries(io, eight, Sq, group, causal):
    case(io, eight, [Sq, Sq + 1, 500, 333], Sq, 2 * group, 2, 16, 64, seed=Sq, causal=causal)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq", [1, 6, 200])
@pytest.mark.parametrize("window,first", [(0, 0), (0, 1), (10, 4), (63, 0), (64, 16), (100, 200), (300, 37), (5000, 4)])
def test_windows_and_first_keys(io, eight, Sq, window, first):
    case(io, eight, [Sq, 250, 900, 1111], Sq, 4, 2, 32, 64, seed=window + first, window=window, first=first)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq", [1, 7, 150])
@pytest.mark.parametrize("kw", [{"softcap": 20.0}, {"slopes": True}, {"sink": True}, {"softcap": 5.0, "slopes": True, "sink": True},
                                {"softcap": 30.0, "window": 50, "first": 3}, {"scale": 0.3, "sink": True, "window": 7}])
def test_modified_scores(io, eight, Sq, kw):
    g = torch.Generator().manual_seed(Sq)
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = 2.0 ** (-torch.arange(1, 7).float())
    if "sink" in kw:
        kw["sink"] = torch.randn(6, generator=g) * 3
        kw["sink"][1] = -math.inf
    case(io, eight, [Sq, 200, 777], Sq, 6, 2, 16, 128, seed=Sq, **kw)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq", [5, 150])
def test_padded_rows_and_rows_without_keys(io, eight, Sq):
    """Query lengths of their own, none among them, and queries before the first position (more rows
    than the cache has keys)."""
    case(io, eight, [300, 400, 60, Sq - 3, 0], Sq, 4, 2, 16, 64, new=[2, Sq, 0, Sq, Sq])
    case(io, eight, [300, 400, 60, 3], Sq, 4, 2, 16, 64, new=[2, Sq, 0, Sq], sink=torch.tensor([0.5, -2.0, 3.0, 0.0]), window=30, first=5)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq", [1, 140])
def test_one_long_sequence(io, eight, Sq):
    """Every share of a long sequence leaves a part, and the parts' references differ."""
    case(io, eight, [40_003], Sq, 4, 2, 64, 128, seed=1, gain=4.0)


@pytest.mark.parametrize("Sq", [1, 140])
def test_scales_far_apart(Sq):
    """Pages whose value scales differ by up to 2^40: each weighted value counts as it is."""
    case(torch.bfloat16, True, [900, 350], Sq, 4, 2, 16, 64, seed=3, spread=20, gain=0.01)


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("Sq", [1, 140])
def test_large_and_growing_scores(io, eight, Sq):
    """Scores of hundreds, whose maximum comes late: references are raised many times."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(2)
    n, P, D, Hkv = 1500, 16, 64, 2
    cache = make_cache(g, 100, Hkv, P, D, E4M3 if eight else io)
    table = torch.arange(94)[None].to(torch.int32)
    ramp = torch.linspace(0.01, 1.0, 94)  # keys grow along the sequence
    if eight:
        cache[2][:94] = (2.0 ** (-10 + torch.arange(94) // 12))[:, None]
    else:
        cache[0][:94] = (cache[0][:94].float() * ramp[:, None, None, None] * 4).to(io)
    q = (torch.randn(1, 4, Sq, D, generator=g) * 6).to(io)
    got = sdpa.sdpa_fwd_cached(q.cuda(), on_gpu(cache), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    check(got, reference(q, cache, table, [n], [Sq]))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("Sq", [1, 3, 140])
def test_same_bits_again_and_in_any_company(eight, Sq):
    """Two calls give the same bits; so do two streams with a workspace each."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(7)
    cache = on_gpu(make_cache(g, 300, 2, 16, 128, E4M3 if eight else torch.bfloat16))
    table = torch.randperm(300, generator=g)[:200].view(2, 100).to(torch.int32).cuda()
    lens = torch.tensor([1500, 777], dtype=torch.int32).cuda()
    q = torch.randn(2, 8, Sq, 128, generator=g).bfloat16().cuda()
    a = sdpa.sdpa_fwd_cached(q, cache, table, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [sdpa.sdpa_fwd_cached(q, cache, table, lens, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, a[0]) and torch.equal(lse, a[1])


@pytest.mark.parametrize("Sq", [1, 40])
def test_workspace_of_the_exact_size_is_not_left(Sq):
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(8)
    cache = on_gpu(make_cache(g, 300, 2, 16, 64, E4M3))
    table = torch.randperm(300, generator=g)[:300].view(1, 300).to(torch.int32).cuda()
    lens = torch.tensor([4800], dtype=torch.int32).cuda()
    q = torch.randn(1, 4, Sq, 64, generator=g).bfloat16().cuda()
    size = sdpa.cached_workspace_size(1, 4, 2, Sq, 64, E4M3, 16, 300)
    buffer = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = sdpa.sdpa_fwd_cached(q, cache, table, lens, workspace=buffer[256:256 + size])
    assert bool((buffer[:256] == 0xA5).all()) and bool((buffer[256 + size:] == 0xA5).all())
    ref = sdpa.sdpa_fwd_cached(q, cache, table, lens)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("Sq", [1, 60])
def test_pages_and_lengths_outside_the_cache(eight, Sq):
    """A page id that the cache does not have: its keys count as not there, and the status says so; a length
    past the table is the table's."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(5)
    cache = make_cache(g, 6, 1, 16, 64, E4M3 if eight else torch.bfloat16)
    q = torch.randn(1, 2, Sq, 64, generator=g).bfloat16()
    for bad in (-1, 6, 1 << 30):
        table = torch.tensor([[0, 3, bad, 2, 5]], dtype=torch.int32)
        got = sdpa.sdpa_fwd_cached(q.cuda(), on_gpu(cache), table.cuda(), torch.tensor([80], dtype=torch.int32).cuda(), causal=False)
        with pytest.raises(sdpa.SdpaError, match="SDPA_ERR_PAGE"):
            sdpa.check_device_status()
        check(got, reference(q, cache, torch.tensor([[0, 3, 2, 5]]), [64], [Sq], causal=False))
    table = torch.tensor([[0, 3, 2, 5]], dtype=torch.int32)
    got = sdpa.sdpa_fwd_cached(q.cuda(), on_gpu(cache), table.cuda(), torch.tensor([9999], dtype=torch.int32).cuda())
    with pytest.raises(sdpa.SdpaError, match="SDPA_ERR_PAGE"):
        sdpa.check_device_status()
    check(got, reference(q, cache, table, [64], [Sq]))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("Sq", [1, 40])
def test_captured_and_replayed_as_the_sequences_grow(eight, Sq):
    """A captured step serves every length that its page table has room for."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(6)
    cache = make_cache(g, 90, 2, 16, 64, E4M3 if eight else torch.float16)
    table = torch.randperm(90, generator=g)[:80].view(2, 40).to(torch.int32)
    gpu, q = on_gpu(cache), torch.randn(2, 4, Sq, 64, generator=g).half().cuda()
    lens, t = torch.tensor([40, 45], dtype=torch.int32).cuda(), table.cuda()
    o, lse = torch.empty_like(q), torch.empty(2, 4, Sq, device="cuda")
    size = sdpa.cached_workspace_size(2, 4, 2, Sq, 64, gpu.k.dtype, 16, 40)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    call = lambda: sdpa.sdpa_fwd_cached(q, gpu, t, lens, o=o, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([40, 45], [64, 65], [333, 40], [640, 639]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(torch.randn(q.shape))
        graph.replay()
        check((o, lse), reference(q.cpu(), cache, table, now, [Sq] * 2))
    sdpa.check_device_status()


@pytest.mark.parametrize("eight", [False, True])
def test_offsets_past_32_bits(eight):
    """A cache of more than 2^32 elements: pages at both its ends."""
    sdpa = _sdpa()
    n_pages, P, D, Hkv = 130, 256, 128, 1032
    raw = torch.zeros(2, n_pages, Hkv, P, D, dtype=torch.uint8 if eight else torch.bfloat16, device="cuda")
    assert raw[0].numel() > 1 << 32
    dtype = E4M3 if eight else torch.bfloat16
    cache = sdpa.KVCache(raw[0].view(dtype), raw[1].view(dtype),
                         *([torch.ones(n_pages, Hkv, device="cuda") for _ in range(2)] if eight else []))
    table = torch.tensor([[129, 0]], dtype=torch.int32).cuda()
    lens = torch.tensor([300], dtype=torch.int32).cuda()
    k, v = (torch.randn(1, Hkv, 300, D, device="cuda").bfloat16() for _ in range(2))
    sdpa.kv_append(k, v, cache, table, lens)
    kd, vd = sdpa.kv_gather(cache, table, lens, 300)
    if not eight:
        assert torch.equal(kd, k) and torch.equal(vd, v)
    q = torch.randn(1, Hkv, 1, D, device="cuda").bfloat16()
    o, lse = sdpa.sdpa_fwd_cached(q, cache, table, lens)
    ref, _ = sdpa.sdpa_fwd(q, kd, vd)
    assert (o.float() - ref.float()).abs().max().item() <= 2.0 ** -6 * vd.abs().max().item()
    sdpa.check_device_status()
