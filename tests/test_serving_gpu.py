"""The cache's operators together, as a serving program and a training step use them (GPU): prompts appended and
attended to, then token by token, then a chunk, over 16- and 8-bit pages; prefixes that sequences share; calls at once on
two streams, on streams given to them and in graphs with one workspace; a layer with positions of several axes."""
import pytest
import torch

import test_given_streams_gpu as given
from cache_reference import positions_of, rotate
from scored_reference import Case, assert_within, doc_ranges
from test_cached_attention_gpu import TYPES, check, reference
from test_kv_cache_gpu import E4M3, on_gpu, make_cache, table_for

pytestmark = pytest.mark.gpu


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def _int(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _cpu(cache):
    return [None if t is None else t.cpu() for t in cache]


@pytest.mark.parametrize("io,eight", TYPES)
@pytest.mark.parametrize("P,D,Hq,Hkv", [(16, 64, 4, 2), (64, 128, 8, 1)])
def test_prompts_tokens_and_a_chunk(io, eight, P, D, Hq, Hkv):
    """Every step's attention against 64 bits over what the cache holds then; at the end the cache's keys and
    values against all that was appended, and sdpa_fwd over what kv_gather reads back against the last step."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(P)
    B, per_row, u = 3, -(-260 // P), torch.finfo(io).eps / 2
    cache = sdpa.kv_cache(B * per_row + 2, Hkv, P, D, dtype=E4M3 if eight else io, device="cuda")
    table = table_for(g, B, per_row, B * per_row + 2)
    freq, lens = sdpa.rope_inv_freq(D), [0] * B
    seen = [[[], []] for _ in range(B)]
    steps = [(100, [100, 37, 81])] + [(1, [1, 1, 1])] * 3 + [(1, [1, 0, 1])] + [(50, [50, 50, 1]), (90, [0, 90, 90])]
    for S, new in steps:
        q, k, v = (torch.randn(B, S, H, D, generator=g).to(io).cuda().transpose(1, 2) for H in (Hq, Hkv, Hkv))
        lens = [n + t for n, t in zip(lens, new)]
        kw = dict(seq_q_lens=None if new == [S] * B else _int(new))
        rq = sdpa.kv_append(k, v, cache, table.cuda(), _int(lens), q=q, inv_freq=freq, **kw)
        o, lse = sdpa.sdpa_fwd_cached(rq, cache, table.cuda(), _int(lens), **kw)
        sdpa.check_device_status()
        check((o, lse), reference(rq.cpu(), _cpu(cache), table, lens, new))
        pos = positions_of(lens, new, S, D // 2)
        for b in range(B):
            for i, t in enumerate((k, v)):
                x = t.cpu()[b:b + 1, :, :new[b]]
                seen[b][i].append(rotate(x, freq.cpu(), pos[b:b + 1, :new[b]])[0] if i == 0 else x.double())
    n = max(lens)
    gk, gv = sdpa.kv_gather(cache, table.cuda(), _int(lens), n, dtype=io)
    for b in range(B):
        for got, parts in zip((gk, gv), seen[b]):
            x, y = torch.cat(parts, 2)[0], got[b, :, :lens[b]].cpu().double()
            assert not got[b, :, lens[b]:].any()
            # One rounding: half a step of the io type (and 2^-20 of the two products, |a| + |b| < 2^4 here). In 8 bits
            # a code, half a step of it (2^-4 of the value, or 2^-10 of a scale: at most 2^-9 |x|max / 448 * 2), which a page
            # whose scale grows by later rows rounds again (2^-10 of the scale again), and the io type's.
            top = x.abs().max().item()
            bound = 2.0 ** -4 * x.abs() + 2 * 2.0 ** -10 * 2 * top / 448 + u * x.abs() * 1.1 if eight else u * x.abs()
            assert ((y - x).abs() - bound - 2.0 ** -16).max().item() <= 0
    # The last step once more, as attention over the plain tensors. Each of the two outputs is off by at most
    # u |O| + u A + 2 e A, A <= |v|max, e <= 2^-23 (D + 16) 20 < 2^-11 (sums |q k| scale up to 20), each LSE by e + 2^-19.
    S, new = steps[-1]
    for b in range(B):
        if new[b] == 0:
            assert not o[b].any() and bool((lse[b] == -float("inf")).all())
            continue
        po, plse = sdpa.sdpa_fwd(rq[b:b + 1, :, :new[b]].contiguous(), gk[b:b + 1, :, :lens[b]].contiguous(),
                                 gv[b:b + 1, :, :lens[b]].contiguous(), causal=True, bottom_right=True)
        vmax = gv[b].float().abs().max().item()
        assert (po.float() - o[b, :, :new[b]].float()).abs().max().item() <= (4 * u + 2.0 ** -9) * vmax
        assert (plse.view(-1) - lse[b, :, :new[b]].reshape(-1)).abs().max().item() <= 2.0 ** -10


@pytest.mark.parametrize("io,eight", TYPES)
def test_a_prefix_that_sequences_share(io, eight):
    """Pages of a prefix in the tables of three sequences: bit for bit what copies of the pages give."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(3)
    B, P, Hq, Hkv, D, prefix = 3, 32, 8, 2, 64, 3
    raw = make_cache(g, 40, Hkv, P, D, E4M3 if eight else io)
    table = table_for(g, B, 6, 30)
    table[:, :prefix] = table[0, :prefix]
    own, copy = table.clone(), on_gpu(raw)
    for b in (1, 2):
        for i in range(prefix):
            own[b, i] = 30 + 3 * (b - 1) + i
            for t in copy:
                if t is not None:
                    t[own[b, i].long()] = t[table[0, i].long()]
    for S in (1, 7, 60):
        k, v = (torch.randn(B, Hkv, S, D, generator=g).to(io).cuda() for _ in range(2))
        q = torch.randn(B, Hq, S, D, generator=g).to(io).cuda()
        lens = _int([prefix * P + S, prefix * P + 20 + S, prefix * P + 32 + S])
        out = []
        for cache, t in ((on_gpu(raw), table), (sdpa.KVCache(*(None if x is None else x.clone() for x in copy)), own)):
            t = t.cuda()
            sdpa.kv_append(k, v, cache, t, lens)
            out.append(sdpa.sdpa_fwd_cached(q, cache, t, lens) + sdpa.kv_gather(cache, t, lens, dtype=io))
        sdpa.check_device_status()
        for a, b in zip(*out):
            assert torch.equal(a, b)


def _state(seed, S, eight, D=64):
    g = torch.Generator().manual_seed(seed)
    raw = make_cache(g, 60, 2, 32, D, E4M3 if eight else torch.bfloat16)
    table, lens = table_for(g, 2, 25, 60).cuda(), _int([700, 333])
    q, k, v = (torch.randn(2, H, S, D, generator=g).bfloat16().cuda() for H in (8, 2, 2))
    return raw, table, lens, q, k, v


def _step(s, cache, freq, **kw):
    _, table, lens, q, k, v = s
    sdpa = _sdpa()
    rq = sdpa.kv_append(k, v, cache, table, lens, q=q, inv_freq=freq, **{a: b for a, b in kw.items() if a == "stream"})
    return sdpa.sdpa_fwd_cached(rq, cache, table, lens, softcap=20.0, **kw)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("S", [1, 5, 40])
def test_two_streams_at_once(S, eight):
    """Two sequences of calls at the same time, on streams given to them: each as alone."""
    sdpa = _sdpa()
    freq = sdpa.rope_inv_freq(64)
    states = [_state(i, S, eight) for i in range(2)]
    want = [_step(s, on_gpu(s[0]), freq) for s in states]
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [[on_gpu(s[0]) for _ in range(10)] for s in states]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(10):
        for j in range(2):
            got[j].append(_step(states[j], caches[j][i], freq, stream=streams[j]))
    torch.cuda.synchronize()
    sdpa.check_device_status()
    for w, many in zip(want, got):
        for one in many:
            assert torch.equal(one[0], w[0]) and torch.equal(one[1], w[1])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("S", [1, 40])
def test_graphs_that_share_a_workspace(S, eight):
    """Two graphs whose calls have one workspace, replayed in turn, with calls outside in between."""
    sdpa = _sdpa()
    freq = sdpa.rope_inv_freq(64)
    states = [_state(i, S, eight) for i in range(2)]
    want = [_step(s, on_gpu(s[0]), freq) for s in states]
    room = torch.empty(sdpa.cached_workspace_size(2, 8, 2, S, 64, E4M3 if eight else torch.bfloat16, 32, 25),
                       dtype=torch.uint8, device="cuda")
    graphs, outs, caches = [], [], [on_gpu(s[0]) for s in states]
    torch.cuda.synchronize()
    for s, c in zip(states, caches):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_step(s, c, freq, workspace=room))
        graphs.append(graph)
    for i in range(4):
        for j in (0, 1):
            for c, raw in zip(caches[j], states[j][0]):
                if c is not None:
                    c.copy_(raw)
            graphs[j].replay()
            if i == 2:
                _step(states[1 - j], on_gpu(states[1 - j][0]), freq, workspace=room)
            assert torch.equal(outs[j][0], want[j][0]) and torch.equal(outs[j][1], want[j][1])


def _given_calls():
    sdpa = _sdpa()
    freq, axes = sdpa.rope_inv_freq(64), sdpa.rope_axes([10, 11, 11])
    calls = {}
    for eight in (False, True):
        s = _state(0, 90, eight)
        cache, (_, table, lens, q, k, v) = on_gpu(s[0]), s
        where = torch.zeros(3, 90, dtype=torch.int32, device="cuda")
        tag = " 8 bits" if eight else ""
        calls["kv_append" + tag] = lambda s, c=cache: (sdpa.kv_append(k, v, c, table, lens, q=q, inv_freq=freq, stream=s),)
        calls["kv_gather" + tag] = lambda s, c=cache: sdpa.kv_gather(c, table, lens, dtype=torch.bfloat16, stream=s)
        calls["sdpa_fwd_cached" + tag] = lambda s, c=cache: sdpa.sdpa_fwd_cached(q, c, table, lens, stream=s)
        calls["one token" + tag] = lambda s, c=cache: sdpa.sdpa_fwd_cached(q[:, :, :1].contiguous(), c, table, lens, stream=s)
    calls["rope axes"] = lambda s: sdpa.rope_fwd(q, k, freq, positions=where, axes=axes, stream=s)
    return calls


GIVEN = [n + t for t in ("", " 8 bits") for n in ("kv_append", "kv_gather", "sdpa_fwd_cached", "one token")] + ["rope axes"]


@pytest.mark.parametrize("name", GIVEN)
def test_outputs_for_given_streams(name, monkeypatch):
    monkeypatch.setattr(given, "_calls", _given_calls)
    given.test_outputs_do_not_take_what_the_current_stream_still_uses(name)
    given.test_outputs_stay_until_both_streams_are_done_with_them(name)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("S", [1, 40])
def test_a_captured_step_on_a_given_stream(S, eight):
    sdpa = _sdpa()
    freq, s = sdpa.rope_inv_freq(64), _state(5, S, eight)
    want = _step(s, on_gpu(s[0]), freq)
    cache, side, graph = on_gpu(s[0]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    room = torch.empty(sdpa.cached_workspace_size(2, 8, 2, S, 64, E4M3 if eight else torch.bfloat16, 32, 25),
                       dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = _step(s, cache, freq, workspace=room, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for c, raw in zip(cache, s[0]):
            if c is not None:
                c.copy_(raw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_axes_than_a_thread_keeps():
    """Six axes, some of them for single pairs: keys and queries of both directions, and the append."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(8)
    sections, B, S, D = (3, 1, 9, 2, 12, 5), 2, 41, 64
    q, k, v = (torch.randn(B, H, S, D, generator=g).bfloat16().cuda() for H in (5, 2, 2))
    axes, freq = sdpa.rope_axes(sections, mixed=True), sdpa.rope_inv_freq(64)
    where = torch.randint(0, 5000, (6, B, S), generator=g, dtype=torch.int32)
    pos = positions_of([S] * B, [S] * B, S, 32, where, axes.cpu())
    for inverse in (False, True):
        fn = sdpa.rope_bwd if inverse else sdpa.rope_fwd
        for got, x in zip(fn(q, k, freq, positions=where.cuda(), axes=axes), (q, k)):
            y, size = rotate(x.cpu(), freq.cpu(), pos * (-1 if inverse else 1))
            assert ((got.cpu().double() - y).abs() - 2.0 ** -8 * y.abs() - size * 2.0 ** -20).max().item() <= 0
    cache, table, lens = sdpa.kv_cache(8, 2, 16, D, dtype=torch.bfloat16, device="cuda"), _int([[7, 1, 2], [3, 4, 5]]), _int([41, 41])
    rq = sdpa.kv_append(k, v, cache, table, lens, q=q, inv_freq=freq, positions=where.cuda(), axes=axes)
    for got, x in ((rq, q), (sdpa.kv_gather(cache, table, lens, S)[0], k)):
        y, size = rotate(x.cpu(), freq.cpu(), pos)
        assert ((got.cpu().double() - y).abs() - 2.0 ** -8 * y.abs() - size * 2.0 ** -20).max().item() <= 0


@pytest.mark.parametrize("D,sections,interleaved,io", [(64, (8, 12, 12), False, torch.bfloat16), (128, (20, 20), True, torch.float16)])
def test_a_layer_with_positions_of_several_axes(D, sections, interleaved, io):
    """Rotation by several axes, attention, and both gradients: stage by stage against 64 bits, the whole step's
    gradients against 64-bit autograd, and against central differences of the 64-bit step."""
    sdpa = _sdpa()
    B, S, Hq, Hkv, rot = 2, 150, 4, 2, 2 * sum(sections)
    case = Case(B, Hq, Hkv, S, S, D, D, io=io, seed=9, softcap=0.0, slopes=None, rows=doc_ranges([[0] * S] * B, None, True, S))
    xq, xk = (t.transpose(1, 2).contiguous() for t in (case.q, case.k))
    f, axes = sdpa.rope_inv_freq(rot), sdpa.rope_axes(sections, mixed=True)
    g = torch.Generator().manual_seed(2)
    where = torch.randint(0, 300, (len(sections), B, S), generator=g, dtype=torch.int32)
    kw = dict(positions=where.cuda(), axes=axes, interleaved=interleaved)
    q, k = sdpa.rope_fwd(xq.cuda().transpose(1, 2), xk.cuda().transpose(1, 2), f, **kw)
    v, do = case.v.cuda(), case.do.cuda()
    o, lse = sdpa.sdpa_fwd(q, k, v, causal=True)
    dq, dk, dv = sdpa.sdpa_bwd(q, k, v, o, do, lse, causal=True)
    gq, gk = (torch.empty_like(t, device="cuda") for t in (xq, xk))
    sdpa.rope_bwd(dq, dk, f, q_out=gq.transpose(1, 2), k_out=gk.transpose(1, 2), **kw)
    sdpa.check_device_status()
    pos = positions_of([S] * B, [S] * B, S, rot // 2, where, axes.cpu())
    u = torch.finfo(io).eps / 2
    tiny = 2.0 ** -25 if io == torch.float16 else 0.0
    for got, x, sign in ((q, xq.transpose(1, 2), 1), (k, xk.transpose(1, 2), 1), (gq.transpose(1, 2), dq, -1), (gk.transpose(1, 2), dk, -1)):
        y, size = rotate(x.cpu(), f.cpu(), pos * sign, interleaved=interleaved)
        assert ((got.cpu().double() - y).abs() - u * y.abs() - size * 2.0 ** -20 - tiny).max().item() <= 0
    # The whole step: q and k rounded shift every score by a random part of sqrt(2) u |score|, |score| up to about 8 here, so
    # P and dS by up to 8 sqrt(2) u relative; O, dS, dQ, dK and the output add a u each: 17 u in the 2-norm.
    x64, k64, v64 = (t.double().requires_grad_(True) for t in (xq, xk, case.v))

    def loss(a, b, c):
        y = _turn(a, f.cpu(), pos, interleaved) @ _turn(b, f.cpu(), pos, interleaved).repeat_interleave(Hq // Hkv, 1).transpose(2, 3) * case.scale
        p = torch.softmax(y.masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), float("-inf")), -1)
        return ((p @ c.repeat_interleave(Hq // Hkv, 1)) * case.do.double()).sum()

    grads = torch.autograd.grad(loss(x64, k64, v64), (x64, k64, v64))
    for name, got, want in zip(("dq", "dk", "dv"), (gq, gk, dv), grads):
        err = (got.cpu().double() - want).norm() / want.norm()
        assert err <= 17 * u, f"{name}: {err:.3e}"
    with torch.no_grad():  # differences along a random direction: off by (1e-4)^2 times third derivatives
        for i, (x, got) in enumerate(zip((x64, k64, v64), (gq, gk, dv))):
            d = torch.randn(x.shape, generator=g, dtype=torch.float64)
            d /= d.norm()
            args = [x64, k64, v64]
            args[i] = x + 1e-4 * d
            up = loss(*args)
            args[i] = x - 1e-4 * d
            along = (up - loss(*args)) / 2e-4
            assert (along - (got.cpu().double() * d).sum()).abs() <= 17 * u * grads[i].norm() + 1e-6 * grads[i].norm()


def _turn(x, f, pos, interleaved):
    """x (B,S,H,D) in 64 bits, turned, as (B,H,S,D) (differentiable)."""
    n = f.numel()
    angle = (pos.double() * f)[:, :, None]
    c, s = angle.cos(), angle.sin()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., 2 * n:]), -1).transpose(1, 2)
