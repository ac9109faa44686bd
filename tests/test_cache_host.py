"""Rotary positions with several axes, the paged cache and attention over it without a GPU: the refusals of the C ABI
(every call here is invalid or has no rows, so nothing is launched), the binding's checks and routes, and pins of the
64-bit reference that the GPU tests use."""
import ctypes
import math
import struct

import pytest
import torch

import attention_backward_sdpa_gb300 as pkg
from cache_reference import code, positions_of, rotate, scale_for
from test_binding_host import _last, fake  # noqa: F401  (the recording library)
from test_scored_host import _taken

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = range(5)
BF16, F16, E4M3 = 0, 2, 3
NAN, INF = float("nan"), float("inf")
# Stand-in pointers, 2^32 bytes apart; never read.
Q, QO, K, V, KC, VC, KS, VS, TABLE, LENS, NEWS, FREQ, POS, AXIS, O, LSE, WS, SINK, SLOPES = ((i + 1) << 32 for i in range(19))


@pytest.fixture(scope="module")
def lib():
    return pkg.load(build_if_missing=True)


# ------------------------------------------------------------------ the C ABI
def _axes(lib, io=BF16, q=Q, k=K, qo=QO, ko=O, B=2, Hq=4, Hkv=2, S=8, D=64, freq=FREQ, rot=64, mult=1.0, pos=POS, per=0,
          n=3, axis=AXIS):
    st = [Hq * S * D, S * D, D] * 2 + [Hkv * S * D, S * D, D] * 2
    return lib.sdpa_rope_axes(io, q, k, qo, ko, B, Hq, Hkv, S, D, (ctypes.c_longlong * 12)(*st), freq, rot, mult, pos, per,
                              n, axis, 0, 0, None)


def test_axes_refusals(lib):
    assert _axes(lib, S=0) == OK
    assert _axes(lib, pos=None) == INVALID and _axes(lib, axis=None) == INVALID
    assert _axes(lib, n=0) == INVALID and _axes(lib, n=-1) == INVALID and _axes(lib, n=17) == INVALID
    assert _axes(lib, axis=AXIS + 2) == ALIGN and _axes(lib, pos=POS + 2) == ALIGN
    assert _axes(lib, io=1) == INVALID and _axes(lib, rot=66) == INVALID and _axes(lib, mult=NAN) == INVALID
    assert _axes(lib, qo=K) == INVALID and _axes(lib, q=Q + 1) == ALIGN


def _append(lib, io=BF16, cache=BF16, q=Q, qo=QO, k=K, v=V, kc=KC, vc=VC, ks=None, vs=None, table=TABLE, lens=LENS,
            news=None, B=2, Hq=4, Hkv=2, S=8, D=64, pages=10, page=16, max_pages=4, strides=None, freq=FREQ, rot=64,
            mult=1.0, pos=None, per=0, n=1, axis=None):
    st = strides or [Hq * S * D, S * D, D] * 2 + [Hkv * S * D, S * D, D] * 2
    return lib.sdpa_kv_append(io, cache, q, qo, k, v, kc, vc, ks, vs, table, lens, news, B, Hq, Hkv, S, D, pages, page,
                              max_pages, (ctypes.c_longlong * 12)(*st), freq, rot, mult, pos, per, n, axis, 0, None)


EIGHT = dict(cache=E4M3, ks=KS, vs=VS)


@pytest.mark.parametrize("call", ["append", "gather", "attention"])
def test_cache_refusals(lib, call):
    """What every call over a cache refuses of it."""
    f = {"append": _append, "gather": _gather, "attention": _attn}[call]
    assert f(lib, S=0) == OK and f(lib, S=0, **EIGHT) == OK
    for kw in (dict(io=1), dict(cache=1), dict(cache=F16), dict(cache=7), dict(io=F16), dict(kc=None), dict(vc=None),
               dict(table=None), dict(lens=None), dict(ks=KS), dict(ks=KS, vs=VS), dict(cache=E4M3),
               dict(cache=E4M3, vs=VS), dict(B=0), dict(Hkv=0), dict(S=-1), dict(D=0), dict(pages=0), dict(max_pages=0),
               dict(pages=1 << 30), dict(max_pages=1 << 27), dict(B=1 << 16, max_pages=1 << 15)):
        assert f(lib, **kw) == INVALID, kw
    for kw in (dict(D=144), dict(D=72), dict(D=8), dict(page=8), dict(page=48), dict(page=512), dict(page=0)):
        assert f(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(kc=KC + 8), dict(vc=VC + 2), dict(table=TABLE + 2), dict(lens=LENS + 1),
               dict(cache=E4M3, ks=KS + 2, vs=VS), dict(cache=E4M3, ks=KS, vs=VS + 1)):
        assert f(lib, **kw) == ALIGN, kw


def test_append_refusals(lib):
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(rot=63), dict(rot=66), dict(rot=-2),
               dict(freq=None), dict(mult=INF), dict(mult=NAN), dict(Hq=-1), dict(axis=AXIS), dict(axis=AXIS, pos=POS, n=0),
               dict(axis=AXIS, pos=POS, n=17), dict(B=1 << 15, S=1 << 14, Hq=8)):
        assert _append(lib, **kw) == INVALID, kw
    for kw in (dict(k=K + 1), dict(v=V + 1), dict(q=Q + 1), dict(qo=QO + 1), dict(freq=FREQ + 4), dict(pos=POS + 2),
               dict(news=NEWS + 2), dict(axis=AXIS + 2, pos=POS, n=2)):
        assert _append(lib, **kw) == ALIGN, kw
    q, kv = [4 * 8 * 64, 8 * 64, 64], [2 * 8 * 64, 8 * 64, 64]
    for out in ([4 * 8 * 64, 8 * 64, 32], [0, 8 * 64, 64], [4 * 8 * 64, 64, 64], [4 * 8 * 64, 8 * 64, -64]):
        assert _append(lib, strides=q + out + kv * 2) == INVALID  # rotated queries over one another
    assert _append(lib, strides=q * 2 + [2 * 8 * 64, -8 * 64, 64] + kv) == INVALID


@pytest.mark.parametrize("eight", [False, True])
def test_append_of_what_overlaps(lib, eight):
    kw = EIGHT if eight else {}
    size = 10 * 2 * 16 * 64 * (1 if eight else 2)  # bytes of a side of the cache
    assert _append(lib, qo=Q + 2, **kw) == INVALID and _append(lib, qo=K, **kw) == INVALID and _append(lib, qo=V, **kw) == INVALID
    for at in (KC, VC):
        for name in ("q", "qo", "k", "v", "table", "lens", "news", "freq", "pos"):
            assert _append(lib, **{**kw, name: at}) == INVALID, name
            assert _append(lib, **{**kw, name: at + size - 16}) == INVALID, name
        assert _append(lib, **{**kw, "axis": at, "pos": POS, "n": 2}) == INVALID
    assert _append(lib, **{**kw, "vc": KC}) == INVALID and _append(lib, **{**kw, "vc": KC + size - 16}) == INVALID
    for name in ("table", "lens", "news", "freq", "pos"):
        assert _append(lib, **{**kw, name: QO}) == INVALID
    if eight:  # one scale for both sides, scales inside the cache or the inputs
        for bad in (dict(vs=KS), dict(vs=KS + 4 * 19), dict(ks=KC), dict(vs=K), dict(ks=QO), dict(ks=Q), dict(vs=TABLE), dict(ks=LENS)):
            assert _append(lib, **{**EIGHT, **bad}) == INVALID, bad


def _gather(lib, io=BF16, cache=BF16, kc=KC, vc=VC, ks=None, vs=None, table=TABLE, lens=LENS, ko=K, vo=V, B=2, Hkv=2, S=8,
            D=64, pages=10, page=16, max_pages=4):
    return lib.sdpa_kv_gather(io, cache, kc, vc, ks, vs, table, lens, ko, vo, B, Hkv, S, D, pages, page, max_pages, None)


def test_gather_refusals(lib):
    for kw in (dict(S=65), dict(B=1 << 16, Hkv=1 << 15, pages=1), dict(ko=None), dict(vo=None), dict(vo=K), dict(vo=K + 2 * 2 * 8 * 64 * 2 - 16), dict(ko=KC),
               dict(vo=VC + 16), dict(ko=TABLE), dict(vo=LENS), dict(cache=E4M3, ks=K, vs=VS), dict(cache=E4M3, ks=KS, vs=V)):
        assert _gather(lib, **kw) == INVALID, kw
    assert _gather(lib, ko=K + 8) == ALIGN and _gather(lib, vo=V + 2) == ALIGN


def _attn(lib, io=BF16, cache=BF16, q=Q, kc=KC, vc=VC, ks=None, vs=None, table=TABLE, lens=LENS, news=None, o=O, lse=LSE,
          B=2, Hq=4, Hkv=2, S=8, D=64, pages=10, page=16, max_pages=4, scale=0.0, window=-1, first=0, sink=None, cap=0.0,
          slopes=None, ws=None, ws_bytes=0):
    return lib.sdpa_fwd_cached(io, cache, q, kc, vc, ks, vs, table, lens, news, o, lse, B, Hq, Hkv, S, D, pages, page,
                               max_pages, scale, 1, window, first, sink, cap, slopes, ws, ws_bytes, None)


def test_attention_refusals(lib):
    need = lib.sdpa_fwd_cached_workspace_size(2, 4, 2, 8, 64, BF16, 16, 4)
    assert need > 0
    for kw in (dict(q=None), dict(o=None), dict(lse=None), dict(Hq=3), dict(Hq=0), dict(first=-1), dict(cap=-1.0),
               dict(cap=NAN), dict(cap=INF), dict(cap=1e-42), dict(B=1 << 10, S=1 << 14, Hq=2, Hkv=2),
               dict(B=1 << 12, S=1, max_pages=1 << 18)):
        assert _attn(lib, **kw) == INVALID, kw
    for kw in (dict(q=Q + 8), dict(o=O + 2), dict(lse=LSE + 2), dict(sink=SINK + 2), dict(slopes=SLOPES + 1),
               dict(news=NEWS + 2), dict(ws=WS + 16, ws_bytes=need)):
        assert _attn(lib, **kw) == ALIGN, kw
    assert _attn(lib, ws=WS, ws_bytes=need - 1) == WORKSPACE
    ws = dict(ws=WS, ws_bytes=need)
    for kw in (dict(o=Q), dict(o=Q + 16), dict(o=KC), dict(o=VC), dict(lse=O), dict(lse=Q), dict(o=TABLE), dict(lse=LENS),
               dict(news=O), dict(sink=LSE), dict(slopes=O), dict(lse=WS, **ws), dict(q=WS, **ws), dict(kc=WS, **ws),
               dict(vc=WS + 256, **ws), dict(cache=E4M3, ks=O, vs=VS), dict(cache=E4M3, ks=KS, vs=LSE)):
        assert _attn(lib, **kw) == INVALID, kw


def test_attention_workspace(lib):
    size = lib.sdpa_fwd_cached_workspace_size
    for bad in ((0, 4, 2, 1, 64, BF16, 16, 4), (1, 3, 2, 1, 64, BF16, 16, 4), (1, 4, 2, 0, 64, BF16, 16, 4),
                (1, 4, 2, 1, 60, BF16, 16, 4), (1, 4, 2, 1, 144, BF16, 16, 4), (1, 4, 2, 1, 64, BF16, 16, 0),
                (1, 4, 2, 1, 64, BF16, 16, 1 << 27)):
        assert size(*bad) == 0
    # Grows with the rows up to what the shares of a device can leave unfinished, then no more.
    one = [size(B, 32, 8, 1, 128, BF16, 64, 512) for B in (1, 2, 64, 1024)]
    assert 0 < one[0] <= one[1] <= one[2] <= one[3] < 64 << 20
    many = [size(1, 32, 8, S, 128, BF16, 64, 512) for S in (9, 500, 5000)]
    assert 0 < many[0] <= many[1] <= many[2] < 64 << 20


# ------------------------------------------------------------------ the binding
def _cache(eight=False, io=torch.bfloat16, pages=10, H=2, page=16, D=64):
    t = torch.float8_e4m3fn if eight else io
    k, v = (torch.zeros(pages, H, page, D).to(t) for _ in range(2))
    return pkg.KVCache(k, v, *((torch.ones(pages, H), torch.ones(pages, H)) if eight else (None, None)))


def _call(B=2, Hq=4, H=2, S=8, D=64, io=torch.bfloat16):
    return (torch.zeros(B, Hq, S, D, dtype=io), torch.zeros(B, H, S, D, dtype=io), torch.zeros(B, H, S, D, dtype=io),
            torch.zeros(B, 4, dtype=torch.int32), torch.full((B,), 8, dtype=torch.int32))


def test_axes_of_pairs():
    a = pkg.rope_axes([2, 3, 3], device="cpu")
    assert a.dtype == torch.int32 and a.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    for bad in ([], [3, -1], [0, 0], [1] * 17):
        with pytest.raises(ValueError):
            pkg.rope_axes(bad, device="cpu")


def test_axes_route(fake):  # noqa: F811
    q, k, *_ = _call()
    f, axes = pkg.rope_inv_freq(64, device="cpu"), pkg.rope_axes([8, 12, 12], device="cpu")
    for pos, per in ((torch.zeros(3, 8, dtype=torch.int32), 0), (torch.zeros(3, 2, 8, dtype=torch.int32), 1)):
        pkg.rope_fwd(q, k, f, positions=pos, axes=axes)
        args = _last(fake, "sdpa_rope_axes")
        assert _taken(fake, "sdpa_rope_axes", args)
        assert args[14:18] == (pos.data_ptr(), per, 3, axes.data_ptr()) and not args[19]
        pkg.rope_bwd(q, k, f, positions=pos, axes=axes)
        assert _last(fake, "sdpa_rope_axes")[19]
    pos, n = torch.zeros(3, 8, dtype=torch.int32), len(fake.calls)
    for kw in (dict(axes=axes), dict(axes=axes.long(), positions=pos), dict(axes=axes[:31], positions=pos),
               dict(axes=axes, positions=pos[:, :7]), dict(axes=axes, positions=pos[0]), dict(axes=axes, positions=pos.long()),
               dict(axes=axes, positions=torch.zeros(3, 1, 8, dtype=torch.int32)), dict(axes=axes, positions=pos, offset=1),
               dict(axes=axes, positions=torch.zeros(17, 8, dtype=torch.int32)), dict(axes=axes, positions=pos[:0])):
        with pytest.raises((ValueError, TypeError)):
            pkg.rope_fwd(q, k, f, **kw)
    assert len(fake.calls) == n


@pytest.mark.parametrize("eight", [False, True])
def test_append_route(fake, eight):  # noqa: F811
    q, k, v, table, lens = _call()
    cache, f = _cache(eight), pkg.rope_inv_freq(32, device="cpu")
    assert pkg.kv_append(k, v, cache, table, lens) is None
    args = _last(fake, "sdpa_kv_append")
    assert _taken(fake, "sdpa_kv_append", args)
    assert args[:2] == (0, E4M3 if eight else BF16) and args[2:4] == (None, None) and args[6:8] == (cache.k.data_ptr(), cache.v.data_ptr())
    assert (args[8] is not None) == eight and args[13:21] == (2, 0, 2, 8, 64, 10, 16, 4)
    rows = q.transpose(1, 2).contiguous().transpose(1, 2)
    got = pkg.kv_append(k, v, cache, table, lens, q=rows, inv_freq=f, mult=1.5, seq_q_lens=lens, interleaved=True)
    args = _last(fake, "sdpa_kv_append")
    assert got.shape == q.shape and got.is_contiguous() and args[12] == lens.data_ptr() and args[14] == 4
    assert struct.unpack("12q", bytes(args[21])) == (2048, 64, 256, 2048, 512, 64, 1024, 512, 64, 1024, 512, 64)
    assert args[22] == f.data_ptr() and args[23] == 32 and args[24] == 1.5 and args[29]
    assert pkg.kv_append(k, v, cache, table, lens, q=q, q_out=q) is q
    pos = torch.zeros(2, 2, 8, dtype=torch.int32)
    pkg.kv_append(k, v, cache, table, lens, inv_freq=f, positions=pos, axes=pkg.rope_axes([8, 8], device="cpu"))
    assert _last(fake, "sdpa_kv_append")[25:28] == (pos.data_ptr(), 1, 2)
    pkg.kv_append(k, v, cache, table, lens, inv_freq=f, positions=pos[0, 0])
    assert _last(fake, "sdpa_kv_append")[25:29] == (pos.data_ptr(), 0, 1, None)


def test_append_argument_checks(fake):  # noqa: F811
    q, k, v, table, lens = _call()
    cache, eight, f = _cache(), _cache(True), pkg.rope_inv_freq(64, device="cpu")
    pos = torch.zeros(8, dtype=torch.int32)
    bad = [((k.float(), v, cache, table, lens), {}), ((k, v.half(), cache, table, lens), {}), ((k[0], v, cache, table, lens), {}),
           ((k, v[:, :1], cache, table, lens), {}), ((k.transpose(2, 3), v.transpose(2, 3), cache, table, lens), {}),
           ((k, None, cache, table, lens), {}), ((k, v, None, table, lens), {}), ((k, v, cache[:2], table, lens), {}),
           ((k, v, _cache(H=1), table, lens), {}), ((k, v, _cache(D=32), table, lens), {}), ((k, v, _cache(io=torch.float16), table, lens), {}),
           ((k, v, cache, table.long(), lens), {}), ((k, v, cache, table[0], lens), {}), ((k, v, cache, table[:1], lens), {}),
           ((k, v, cache, table, lens.long()), {}), ((k, v, cache, table, lens[:1]), {}), ((k, v, cache, None, lens), {}),
           ((k, v, cache._replace(k_scale=torch.ones(10, 2)), table, lens), {}), ((k, v, eight._replace(v_scale=None), table, lens), {}),
           ((k, v, eight._replace(v_scale=torch.ones(10, 1)), table, lens), {}), ((k, v, eight._replace(v_scale=torch.ones(10, 2).half()), table, lens), {}),
           ((k, v, cache._replace(v=cache.v[:9]), table, lens), {}), ((k, v, cache._replace(v=cache.v.transpose(2, 3)), table, lens), {})]
    bad += [((k, v, cache, table, lens), kw) for kw in (
        dict(q=q[0]), dict(q=q[:1]), dict(q=q.half()), dict(q_out=q), dict(q=q, q_out=q[:, :2]), dict(q=q, q_out=q.half()),
        dict(seq_q_lens=lens[:1]), dict(seq_q_lens=lens.long()), dict(inv_freq=f.float()), dict(inv_freq=f[:0]),
        dict(inv_freq=torch.zeros(33, dtype=torch.float64)), dict(positions=pos), dict(axes=pos), dict(inv_freq=f, positions=pos[:7]),
        dict(inv_freq=f, positions=pos.long()), dict(inv_freq=f, axes=torch.zeros(32, dtype=torch.int32)),
        dict(inv_freq=f, positions=pos[None], axes=torch.zeros(31, dtype=torch.int32)))]
    for a, kw in bad:
        with pytest.raises((ValueError, TypeError)):
            pkg.kv_append(*a, **kw)
    assert not fake.calls


def test_gather_route(fake):  # noqa: F811
    *_, table, lens = _call()
    for cache, dtype, want in ((_cache(), None, torch.bfloat16), (_cache(True), None, torch.bfloat16), (_cache(True), torch.float16, torch.float16),
                               (_cache(io=torch.float16), None, torch.float16)):
        k, v = pkg.kv_gather(cache, table, lens, dtype=dtype)
        args = _last(fake, "sdpa_kv_gather")
        assert _taken(fake, "sdpa_kv_gather", args) and args[10:17] == (2, 2, 64, 64, 10, 16, 4)
        assert k.shape == v.shape == (2, 2, 64, 64) and k.dtype == v.dtype == want
    out = torch.zeros(2, 2, 5, 64, dtype=torch.bfloat16)
    assert pkg.kv_gather(_cache(), table, lens, 5, k_out=out, v_out=out.clone())[0] is out
    n = len(fake.calls)
    for a, kw in (((_cache(), table, lens, 65), {}), ((_cache(), table, lens, -1), {}), ((_cache(), table, lens, 2.5), {}),
                  ((_cache(), table, lens), dict(dtype=torch.float16)), ((_cache(), table, lens), dict(dtype=torch.float32)),
                  ((_cache(), table, lens), dict(k_out=out)), ((_cache(), table, lens, 5), dict(v_out=out.half())),
                  ((None, table, lens), {}), ((_cache(), table[0], lens), {}), ((_cache(), table, lens[:1]), {})):
        with pytest.raises((ValueError, TypeError)):
            pkg.kv_gather(*a, **kw)
    assert len(fake.calls) == n


@pytest.mark.parametrize("eight", [False, True])
def test_attention_route(fake, eight, monkeypatch):  # noqa: F811
    monkeypatch.setattr(pkg, "_cached_workspace", lambda *a: 512)
    q, _, _, table, lens = _call()
    cache = _cache(eight)
    o, lse = pkg.sdpa_fwd_cached(q, cache, table, lens)
    args = _last(fake, "sdpa_fwd_cached")
    assert _taken(fake, "sdpa_fwd_cached", args)
    assert args[:2] == (0, E4M3 if eight else BF16) and args[12:20] == (2, 4, 2, 8, 64, 10, 16, 4)
    assert args[20:24] == (0.0, 1, -1, 0) and args[-2] == 512 and o.shape == q.shape and lse.shape == (2, 4, 8)
    sink, slopes = torch.zeros(4), torch.ones(4)
    pkg.sdpa_fwd_cached(q, cache, table, lens, scale=0.5, causal=False, window_left=7, first_keys=3, sink=sink, softcap=9.0,
                        alibi_slopes=slopes, seq_q_lens=lens, o=o, lse=lse, workspace=torch.zeros(1024, dtype=torch.uint8))
    args = _last(fake, "sdpa_fwd_cached")
    assert args[9] == lens.data_ptr() and args[10:12] == (o.data_ptr(), lse.data_ptr()) and args[20:24] == (0.5, 0, 7, 3)
    assert args[24:27] == (sink.data_ptr(), 9.0, slopes.data_ptr()) and args[-2] == 1024
    n = len(fake.calls)
    for a, kw in (((q[0], cache, table, lens), {}), ((q.float(), cache, table, lens), {}), ((q.half(), cache, table, lens), {} if not eight else dict(sink=sink[:1])),
                  ((q.transpose(1, 2), cache, table, lens), {}), ((q[..., :32].contiguous(), cache, table, lens), {}),
                  ((q, cache, table[:1], lens), {}), ((q, cache, table, lens), dict(seq_q_lens=lens[:1])),
                  ((q, cache, table, lens), dict(sink=sink[:3])), ((q, cache, table, lens), dict(softcap=-1.0)),
                  ((q, cache, table, lens), dict(softcap=math.inf)), ((q, cache, table, lens), dict(alibi_slopes=slopes[:3])),
                  ((q, cache, table, lens), dict(window_left=1.5)), ((q, cache, table, lens), dict(first_keys=-1)),
                  ((q, cache, table, lens), dict(window_left=1 << 31)), ((q, cache, table, lens), dict(o=o.half())),
                  ((q, cache, table, lens), dict(lse=lse[:1])), ((q, cache, table, lens), dict(workspace=torch.zeros(8, 200, dtype=torch.uint8).T))):
        with pytest.raises((ValueError, TypeError)):
            pkg.sdpa_fwd_cached(*a, **kw)
    assert len(fake.calls) == n


def test_kv_cache_of_a_size():
    for eight in (False, True):
        c = pkg.kv_cache(5, 2, 16, 64, dtype=torch.float8_e4m3fn if eight else torch.float16, device="cpu")
        assert c.k.shape == c.v.shape == (5, 2, 16, 64) and c.k.dtype == (torch.float8_e4m3fn if eight else torch.float16)
        assert not c.k.float().any() and not c.v.float().any()
        assert (c.k_scale is None) == (c.v_scale is None) == (not eight)
        if eight:
            assert c.k_scale.shape == (5, 2) and bool((c.k_scale > 0).all()) and c.k_scale.data_ptr() != c.v_scale.data_ptr()
    for bad in (dict(page_size=24), dict(page_size=512), dict(D=72), dict(D=144), dict(dtype=torch.float32), dict(n_pages=0)):
        kw = {**dict(n_pages=5, Hkv=2, page_size=16, D=64), **bad}
        with pytest.raises(ValueError):
            pkg.kv_cache(kw.pop("n_pages"), kw.pop("Hkv"), kw.pop("page_size"), kw.pop("D"), device="cpu", **kw)


# ------------------------------------------------------------------ the reference
def test_codes_of_the_reference():
    """Every finite code is itself, every middle goes to the even one, and what torch rounds agrees in range."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    fin = every[every.isfinite()]
    assert torch.equal(code(fin), fin)
    pos = fin[fin >= 0].sort().values.unique()
    mid = (pos[:-1] + pos[1:]) / 2
    down, up = pos[:-1], pos[1:]
    even = torch.where(torch.arange(len(mid)) % 2 == 0, down, up)  # (codes in order: every second one is even)
    assert torch.equal(code(mid), even) and torch.equal(code(-mid), -even)
    assert torch.equal(code(mid * (1 + 1e-9)), up) and torch.equal(code(mid * (1 - 1e-9)), down)
    assert code(torch.tensor([1e9, -math.inf, math.nan], dtype=torch.float64)).nan_to_num(nan=7.0).tolist() == [448.0, -448.0, 7.0]
    x = torch.randn(10000, generator=torch.Generator().manual_seed(0)) * 50
    assert torch.equal(code(x.double()), x.to(torch.float8_e4m3fn).float().double())


def test_scales_of_the_reference():
    for e in (-70, -64, -60, -1, 0, 5, 100):
        top = 448.0 * 2.0 ** e
        assert scale_for(top) == 2.0 ** max(e, -64)
        assert scale_for(top * (1 + 2.0 ** -20)) == 2.0 ** max(e + 1, -64)
        assert scale_for(top * (1 - 2.0 ** -20)) == 2.0 ** max(e, -64)
    assert scale_for(0.0) == 2.0 ** -64


def test_rotation_of_the_reference():
    """A rotation by complex numbers, and positions that the cache gives."""
    g = torch.Generator().manual_seed(1)
    x, f = torch.randn(2, 3, 5, 16, generator=g, dtype=torch.float64), torch.rand(4, generator=g, dtype=torch.float64)
    pos = positions_of([9, 30], [3, 5], 5, 4)
    assert pos.shape == (2, 5, 4) and pos[0, :, 0].tolist() == [6, 7, 8, 9, 10] and pos[1, 0].tolist() == [25] * 4
    turn = torch.polar(torch.ones(2, 5, 4, dtype=torch.float64), pos * f)[:, None]
    y, size = rotate(x, f, pos, 1.5)
    z = torch.complex(x[..., :4], x[..., 4:8]) * turn * 1.5
    assert (y[..., :4] - z.real).abs().max() < 1e-14 and (y[..., 4:8] - z.imag).abs().max() < 1e-14
    assert torch.equal(y[..., 8:], x[..., 8:]) and not size[..., 8:].any()
    y, _ = rotate(x, f, pos, 1.0, interleaved=True)
    z = torch.complex(x[..., 0:8:2], x[..., 1:8:2]) * turn
    assert (y[..., 0:8:2] - z.real).abs().max() < 1e-14 and (y[..., 1:8:2] - z.imag).abs().max() < 1e-14
    axes = torch.tensor([1, 0, 0, 1], dtype=torch.int32)
    p = torch.arange(20, dtype=torch.int32).view(2, 2, 5)
    got = positions_of([9, 30], [3, 5], 5, 4, p, axes)
    assert torch.equal(got[..., 0], p[1].long()) and torch.equal(got[..., 2], p[0].long())
