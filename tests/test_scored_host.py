"""Modified scores, mask plans and the rotary embedding without a GPU: the refusals of
the C ABI (every call here is invalid, so nothing is launched), the binding's checks and
routes, and pins of the 64-bit reference that the GPU tests use: float64 autograd and
central differences."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import attention_backward_sdpa_gb300 as pkg
from scored_reference import Case, doc_ranges, visible
from test_binding_host import _last, fake  # noqa: F401  (the recording library)
from test_scored_limits_gpu import fp16_bound

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = range(5)
P = 1 << 20  # a stand-in pointer, 256-byte aligned; never read (every call is refused)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return pkg.load(build_if_missing=True)


# ------------------------------------------------------------------ the C ABI
def _fwd(lib, softcap=20.0, slopes=None, plan=None, io=0, scale=0.0, B=1, Hq=2, Hkv=2, Sq=64, Skv=64, Dqk=64, Dv=64,
         q=P, causal=0, wr=-1):
    return lib.sdpa_fwd_scored(io, q, P, P, P, P, B, Hq, Hkv, Sq, Skv, Dqk, Dv, scale, causal, 0, -1, wr, None, None,
                               None, softcap, slopes, plan, None)


def _bwd(lib, softcap=20.0, slopes=None, plan=None, io=0, det=0, D=64, sink=None, dsink=None, ws=None, ws_bytes=0,
         Hkv=2, causal=0, wr=-1):
    return lib.sdpa_bwd_scored(io, P, P, P, P, P, P, P, P, P, 1, 2, Hkv, 64, 64, D, D, 0.0, causal, 0, -1, wr, det,
                               None, None, ws, ws_bytes, sink, dsink, softcap, slopes, plan, None)


@pytest.mark.parametrize("softcap", [-1.0, NAN, INF, -INF])
def test_caps_that_are_refused(lib, softcap):
    assert _fwd(lib, softcap=softcap) == INVALID
    assert _bwd(lib, softcap=softcap) == INVALID


def test_caps_below_fp32s_normal_numbers(lib, fake):  # noqa: F811
    """A cap that rounds to 0 in fp32 would be no cap at all."""
    assert _fwd(lib, softcap=1e-39, scale=1e-30) == INVALID and _bwd(lib, softcap=1e-39) == INVALID
    q, k, v, o, do, lse = _cpu()
    for softcap in (5e-324, 1e-60, 2.0 ** -127):
        with pytest.raises(ValueError):
            pkg.sdpa_fwd(q, k, v, softcap=softcap)
        with pytest.raises(ValueError):
            pkg.sdpa_bwd(q, k, v, o, do, lse, softcap=softcap)
    assert not fake.calls


def test_cap_far_from_the_scale(lib):
    """scale / cap or cap * log2(e) outside fp32's normal range."""
    assert _fwd(lib, softcap=1e-38, scale=100.0) == INVALID       # the ratio overflows
    assert _fwd(lib, softcap=3e38, scale=1e-3) == INVALID         # it is subnormal
    assert _fwd(lib, softcap=3.4e38, scale=100.0) == INVALID      # the cap in log2 units overflows


def test_refusals_of_the_scored_calls(lib):
    for call in (_fwd, _bwd):
        assert call(lib, io=1) == INVALID and call(lib, io=7) == INVALID
        assert call(lib, slopes=P + 2) == ALIGN
        assert call(lib, plan=P + 128) == ALIGN
        assert call(lib, wr=3) == UNSUPPORTED                     # a right band needs causal
    assert _fwd(lib, q=None) == INVALID and _fwd(lib, q=P + 8) == ALIGN
    assert _fwd(lib, Hkv=3) == INVALID
    assert _fwd(lib, Dqk=72, Dv=64) == UNSUPPORTED and _fwd(lib, Dqk=160, Dv=160) == UNSUPPORTED
    assert _fwd(lib, plan=P, Skv=0) == INVALID and _fwd(lib, plan=P, Sq=0) == INVALID
    assert _bwd(lib, dsink=P) == INVALID                          # dsink without a sink
    # The ordered relay does not take a plan; the stored-dS route (D 128 and above) does.
    assert _bwd(lib, plan=P, det=1, D=64) == UNSUPPORTED
    assert _bwd(lib, plan=P, det=1, D=80) == UNSUPPORTED


def test_scored_workspace_size(lib):
    """The plain size plus two more bytes per element of the per-head partials."""
    a256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for B, Hq, Hkv, Sq, Skv, D, det in ((2, 8, 2, 100, 130, 64, 0), (1, 4, 1, 64, 64, 128, 1), (1, 6, 3, 300, 77, 256, 0)):
        args = (B, Hq, Hkv, Sq, Skv, D, D, 1, 0, -1, -1, det, 0)
        part = B * Hq * Skv * D
        assert lib.sdpa_bwd_scored_workspace_size(*args) - lib.sdpa_bwd_workspace_size(*args) \
            == 2 * (a256(4 * part) - a256(2 * part))
        same = (B, Hq, Hq) + args[3:]
        assert lib.sdpa_bwd_scored_workspace_size(*same) == lib.sdpa_bwd_workspace_size(*same)
        assert pkg.workspace_size(B, Hq, Hkv, Sq, Skv, D, D, bool(det), causal=True, scored=True) \
            == lib.sdpa_bwd_scored_workspace_size(*args)
    assert lib.sdpa_bwd_scored_workspace_size(1, 4, 3, 64, 64, 64, 64, 0, 0, -1, -1, 0, 0) == 0


def test_mask_plan_refusals(lib):
    size = lib.sdpa_mask_plan_size
    n = size(2, 100, 300)
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    # ranges, query-tile and key-tile summaries, rows per key, one flag per batch row
    assert n == up(2 * 128 * 8) + up(2 * 2 * 16) + up(2 * 3 * 8) + up(2 * 384 * 8 + 2 * 4)
    for bad in ((0, 64, 64), (1, 0, 64), (1, 64, 0), (-1, 64, 64), (1 << 20, 1 << 11, 64), (4, 64, 1 << 29)):
        assert size(*bad) == 0
    rows, docs = lib.sdpa_mask_plan_rows, lib.sdpa_mask_plan_docs
    assert rows(None, P, 2, 100, 300, P, n, None) == INVALID and rows(P, None, 2, 100, 300, P, n, None) == INVALID
    assert rows(P, P, 2, 100, 300, None, n, None) == INVALID
    assert rows(P, P, 0, 100, 300, P, n, None) == INVALID
    assert rows(P + 2, P, 2, 100, 300, P, n, None) == ALIGN and rows(P, P, 2, 100, 300, P + 64, n, None) == ALIGN
    assert rows(P, P, 2, 100, 300, P, n - 1, None) == WORKSPACE
    m = size(2, 100, 100)
    assert docs(P, P, 0, 0, 2, 100, P, m, None) == INVALID        # a prefix without causal
    assert docs(P, None, 0, 1, 2, 100, P, m - 1, None) == WORKSPACE
    assert docs(P + 1, None, 0, 1, 2, 100, P, m, None) == ALIGN
    assert docs(P, P + 2, 0, 1, 2, 100, P, m, None) == ALIGN
    assert docs(P, None, 0, 1, 2, 0, P, m, None) == INVALID


def _rope(lib, io=0, q=P, k=P, qo=P, ko=P, B=2, Hq=4, Hkv=2, S=8, D=64, strides=None, freq=P, rot=64, mult=1.0,
          pos=None, per=0, offset=0):
    st = strides or [Hq * S * D, S * D, D] * 2 + [Hkv * S * D, S * D, D] * 2
    return lib.sdpa_rope(io, q, k, qo, ko, B, Hq, Hkv, S, D, (ctypes.c_longlong * 12)(*st), freq, rot, mult, pos, per,
                         offset, 0, 0, None)


def test_rope_refusals(lib):
    assert _rope(lib, io=1) == INVALID
    assert _rope(lib, q=None) == INVALID and _rope(lib, k=None) == INVALID and _rope(lib, ko=None) == INVALID
    assert _rope(lib, freq=None) == INVALID
    assert _rope(lib, rot=0) == INVALID and _rope(lib, rot=63) == INVALID and _rope(lib, rot=66) == INVALID
    assert _rope(lib, D=1024, rot=514) == UNSUPPORTED
    assert _rope(lib, mult=NAN) == INVALID and _rope(lib, mult=INF) == INVALID
    assert _rope(lib, Hq=0) == INVALID and _rope(lib, S=-1) == INVALID and _rope(lib, B=0) == INVALID
    assert _rope(lib, S=0) == OK
    assert _rope(lib, q=P + 1) == ALIGN and _rope(lib, freq=P + 4) == ALIGN and _rope(lib, pos=P + 2) == ALIGN
    assert _rope(lib, offset=-1) == INVALID and _rope(lib, offset=(1 << 31) - 7) == INVALID
    assert _rope(lib, B=1 << 14, S=1 << 14, Hq=8) == INVALID      # 2^31 rows or more
    plain = [4 * 8 * 64, 8 * 64, 64]
    kv = [2 * 8 * 64, 8 * 64, 64] * 2
    for out in ([4 * 8 * 64, 8 * 64, 32], [4 * 8 * 64, 64, 64], [0, 8 * 64, 64], [4 * 8 * 64, -8 * 64, 64],
                [8 * 64, 8 * 64, 64]):
        assert _rope(lib, strides=plain + out + kv) == INVALID    # output rows overlap
    assert _rope(lib, strides=[4 * 8 * 64, -8 * 64, 64] + plain + kv) == INVALID  # a negative input stride


def test_rope_outputs_that_overlap(lib):
    """An output shares elements with its own input alone, one for one (all refused: nothing runs)."""
    B, Hq, Hkv, S, D = 2, 4, 2, 8, 64
    far = [P + (i << 20) for i in range(4)]  # q, k, q_out, k_out apart from each other

    def call(strides=None, **at):
        ptr = dict(zip(("q", "k", "qo", "ko"), far))
        ptr.update(at)
        return _rope(lib, strides=strides, **ptr)

    row = 2 * D
    assert call(qo=far[0] + row) == INVALID and call(qo=far[0] + 16) == INVALID     # q, a row or less further on
    assert call(qo=far[0] + (B * Hq * S - 1) * row) == INVALID                      # its last row
    assert call(qo=far[1]) == INVALID and call(ko=far[0]) == INVALID                # the other input
    assert call(ko=far[2]) == INVALID and call(ko=far[2] + 5 * row) == INVALID      # the other output
    plain, turned = [Hq * S * D, S * D, D], [S * Hq * D, D, Hq * D]                 # (B, H, S, D) and (B, S, H, D)
    kv = [Hkv * S * D, S * D, D] * 2
    assert call(strides=plain + turned + kv, qo=far[0]) == INVALID                  # in place, but rows change places
    assert call(strides=turned + plain + kv, qo=far[0]) == INVALID
    # A projection's row of Hq + Hkv + Hkv heads: each tensor a slice; the keys one head too low meet the queries.
    width = (Hq + 2 * Hkv) * D
    fused = [S * width, D, width]
    assert call(strides=fused * 4, q=far[0], qo=far[0], k=far[0] + Hq * row, ko=far[0] + (Hq - 1) * row) == INVALID
    assert call(strides=fused * 4, q=far[0], qo=far[0] + Hkv * row, k=far[1], ko=far[3]) == INVALID
    # The same places with other strides: not followed row by row.
    assert call(strides=fused * 2 + fused + [S * width, D, 2 * width], q=far[0], qo=far[0], k=far[0] + Hq * row,
                ko=far[0] + (Hq + Hkv) * row) == INVALID


# ------------------------------------------------------------------ the binding
def _cpu(B=2, Hq=4, Hkv=2, S=96, D=64, io=torch.bfloat16):
    q, k = torch.zeros(B, Hq, S, D, dtype=io), torch.zeros(B, Hkv, S, D, dtype=io)
    return q, k, k.clone(), q.clone(), q.clone(), torch.zeros(B, Hq, S)


def test_scored_routes(fake):  # noqa: F811
    q, k, v, o, do, lse = _cpu()
    slopes = torch.zeros(4)
    plan = pkg.MaskPlan(2, 96, 96, torch.zeros(8, dtype=torch.uint8))
    for kw in (dict(softcap=30.0), dict(alibi_slopes=slopes), dict(mask_plan=plan),
               dict(softcap=5.0, alibi_slopes=slopes, mask_plan=plan)):
        pkg.sdpa_fwd(q, k, v, causal=True, **kw)
        args = _last(fake, "sdpa_fwd_scored")
        assert args[0] == 0 and args[6:13] == (2, 4, 2, 96, 96, 64, 64) and args[-4] == kw.get("softcap", 0.0)
        out = pkg.sdpa_bwd(q, k, v, o, do, lse, causal=True, **kw)
        _last(fake, "sdpa_bwd_scored")
        assert len(out) == 3
    sink = torch.zeros(4)
    assert len(pkg.sdpa_bwd(q, k, v, o, do, lse, sink=sink, softcap=1.0)) == 4
    pkg.sdpa_fwd(q.half(), k.half(), v.half(), softcap=2.0)
    assert _last(fake, "sdpa_fwd_scored")[0] == 2
    pkg.sdpa_fwd(q, k, v, softcap=0.0)
    _last(fake, "sdpa_fwd")


def test_numpy_scalars(fake):  # noqa: F811
    """The scored and rotary calls take the numbers that the plain calls take."""
    q, k, v, o, do, lse = _cpu()
    kw = dict(scale=np.float32(0.125), causal=np.bool_(True), bottom_right=np.bool_(False), window_left=np.int64(40),
              window_right=np.int32(3), softcap=np.float32(30.0))
    pkg.sdpa_fwd(q, k, v, **kw)
    args = _last(fake, "sdpa_fwd_scored")
    assert _taken(fake, "sdpa_fwd_scored", args)
    pkg.sdpa_bwd(q, k, v, o, do, lse, deterministic=np.bool_(True), **kw)
    assert _taken(fake, "sdpa_bwd_scored", _last(fake, "sdpa_bwd_scored"))
    size = [a for n, a in fake.calls if n == "sdpa_bwd_scored_workspace_size"]
    assert len(size) == 1 and _taken(fake, "sdpa_bwd_scored_workspace_size", size[0])
    f = pkg.rope_inv_freq(64, device="cpu")
    pkg.rope_fwd(q, k, f, mult=np.float32(1.5), offset=np.int64(7), interleaved=np.bool_(True))
    assert _taken(fake, "sdpa_rope", _last(fake, "sdpa_rope"))
    with pytest.raises(TypeError):
        pkg.rope_fwd(q, k, f, offset=1.5)


def _taken(fake, name, args):  # noqa: F811
    """Whether ctypes takes the arguments as declared (nothing is called)."""
    for kind, a in zip(getattr(fake.real, name).argtypes, args):
        kind.from_param(a)
    return True


def test_scored_argument_checks(fake):  # noqa: F811
    q, k, v, o, do, lse = _cpu()
    plan = pkg.MaskPlan(2, 96, 95, torch.zeros(8, dtype=torch.uint8))
    bias = torch.zeros(1, 4, 96, 96)
    for kw, err in ((dict(softcap=-1.0), ValueError), (dict(softcap=NAN), ValueError), (dict(softcap=INF), ValueError),
                    (dict(alibi_slopes=torch.zeros(3)), ValueError),
                    (dict(alibi_slopes=torch.zeros(4, dtype=torch.float64)), ValueError),
                    (dict(alibi_slopes=torch.zeros(8)[::2]), ValueError), (dict(alibi_slopes=[1.0] * 4), ValueError),
                    (dict(mask_plan=plan), ValueError), (dict(mask_plan=torch.zeros(8)), TypeError),
                    (dict(softcap=2.0, bias=bias), ValueError), (dict(softcap=2.0, window_left=1 << 32), ValueError),
                    (dict(softcap=2.0, causal=True, window_right=1 << 31), ValueError)):
        with pytest.raises(err):
            pkg.sdpa_fwd(q, k, v, **kw)
        with pytest.raises(err):
            pkg.sdpa_bwd(q, k, v, o, do, lse, **kw)
    assert not fake.calls


def test_mask_plan_argument_checks(fake):  # noqa: F811
    ids = torch.zeros(2, 96, dtype=torch.int32)
    pre = torch.zeros(2, dtype=torch.int32)
    for kw in (dict(Skv=95, doc_ids=ids), dict(doc_ids=ids.long()), dict(doc_ids=ids[:, :95]),
               dict(doc_ids=ids, prefix_lens=pre), dict(doc_ids=ids, prefix_lens=ids[:1], causal=True),
               dict(row_lo=ids), dict(row_lo=ids, row_hi=ids, causal=True), dict(row_lo=ids, row_hi=ids, doc_ids=ids),
               dict(row_lo=ids.t().contiguous().t(), row_hi=ids)):
        with pytest.raises(ValueError):
            pkg.mask_plan(2, 96, kw.pop("Skv", 96), **kw)
    for sizes in ((0, 96, 96), (2, -1, -1), ((1 << 32) + 1, 96, 96), (1, 1 << 31, 1 << 31)):
        with pytest.raises(ValueError):
            pkg.mask_plan(*sizes, causal=True)
    assert not [c for c in fake.calls if c[0] != "sdpa_mask_plan_size"]


def test_rope_argument_checks(fake):  # noqa: F811
    q, k = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    f = pkg.rope_inv_freq(64, device="cpu")
    pkg.rope_fwd(q, k, f)
    assert _last(fake, "sdpa_rope")[0] == 0
    assert list(struct.unpack("12q", _last(fake, "sdpa_rope")[10])) == [4096, 1024, 64] * 2 + [2048, 1024, 64] * 2
    pkg.rope_bwd(q.transpose(1, 2).contiguous().transpose(1, 2), None, f[:8].contiguous(), interleaved=True,
                 positions=torch.zeros(16, dtype=torch.int32))
    args = _last(fake, "sdpa_rope")
    st = list(struct.unpack("12q", args[10]))
    assert st[:6] == [4096, 64, 256, 4096, 1024, 64] and args[7] == 0 and args[12] == 16
    assert args[15] == 0 and args[-3:-1] == (True, True)
    n = len(fake.calls)
    pos = torch.zeros(2, 16, dtype=torch.int32)
    for a, kw in (((q.float(), k, f), {}), ((q, k.half(), f), {}), ((q, k, f.float()), {}), ((q, k, f[None]), {}),
                  ((q, k, torch.zeros(33, dtype=torch.float64)), {}), ((q, k, f[:0]), {}),
                  ((q, k[:1], f), {}), ((q, k[:, :, :15], f), {}), ((q[0], k, f), {}), ((q, k[0], f), {}),
                  ((q.transpose(2, 3), None, f[:8]), {}), ((q, k, f), dict(positions=pos.long())),
                  ((q, k, f), dict(positions=pos[:, :15])), ((q, k, f), dict(positions=pos, offset=3)),
                  ((q, k, f), dict(offset=-1)), ((q, k, f), dict(offset=(1 << 31) - 15)), ((q, k, f), dict(offset=1 << 32)),
                  ((q, None, f), dict(k_out=k)), ((q, k, f), dict(q_out=k)), ((q, k, f), dict(q_out=q.half()))):
        with pytest.raises((ValueError, TypeError)):
            pkg.rope_fwd(*a, **kw)
    assert len(fake.calls) == n


def test_rope_of_keys_alone(fake):  # noqa: F811
    """Without query heads the keys are the call's first tensor; without any head there is no call."""
    q, k = torch.zeros(2, 0, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 16, 64, dtype=torch.bfloat16)
    f = pkg.rope_inv_freq(64, device="cpu")
    yq, yk = pkg.rope_fwd(q, k.transpose(1, 2).contiguous().transpose(1, 2), f)
    args = _last(fake, "sdpa_rope")
    assert args[2] is None and args[3] == yk.data_ptr() and args[4] is None and args[5:10] == (2, 3, 0, 16, 64)
    assert list(struct.unpack("12q", args[10]))[:6] == [3072, 64, 192, 3072, 1024, 64]
    assert yq.shape == q.shape and yk.shape == k.shape
    n = len(fake.calls)
    pkg.rope_fwd(q, q, f), pkg.rope_fwd(q, None, f), pkg.rope_fwd(k[:0], k[:0], f)
    assert len(fake.calls) == n


def test_inverse_frequencies():
    f = pkg.rope_inv_freq(8, 100.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 100.0 ** -0.25, 0.1, 100.0 ** -0.75], dtype=torch.float64), rtol=1e-15)
    assert torch.equal(pkg.rope_inv_freq(8, 100.0, scaling="linear", factor=4.0, device="cpu"), f / 4)
    n = pkg.rope_inv_freq(8, 100.0, scaling="ntk", factor=4.0, device="cpu")
    assert n[0] == 1.0 and math.isclose(n[-1], f[-1] / 4, rel_tol=1e-14)  # highest kept, lowest / factor
    b = pkg.rope_inv_freq(64, 10000.0, scaling="bands", factor=8.0, original_len=4096, device="cpu")
    g = pkg.rope_inv_freq(64, 10000.0, device="cpu")
    turns = 4096 * g / (2 * math.pi)
    assert torch.equal(b[turns >= 32], g[turns >= 32]) and torch.equal(b[turns <= 1], g[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((b[mid] < g[mid]) & (b[mid] > g[mid] / 8)).all()
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, base=-1.0), dict(rot_dim=8, factor=0.0),
                dict(rot_dim=8, scaling="other"), dict(rot_dim=2, scaling="ntk"), dict(rot_dim=8, scaling="bands")):
        with pytest.raises(ValueError):
            pkg.rope_inv_freq(device="cpu", **bad)


# ------------------------------------------------------------------ the reference
def test_document_ranges_by_hand():
    assert doc_ranges([[4, 4, 9, 9, 9, 4]], None, False, 6) == [[(0, 2), (0, 2), (2, 5), (2, 5), (2, 5), (5, 6)]]
    assert doc_ranges([[4, 4, 9, 9, 9, 4]], [2], True, 6) == [[(0, 2), (0, 2), (2, 4), (2, 4), (2, 5), (5, 6)]]


CASES = [dict(softcap=3.0, causal=True), dict(slopes=[0.5, -0.1], bottom_right=True, causal=True),
         dict(softcap=1.5, slopes=[0.2, 0.0], rows="some", window_left=9),
         dict(rows="some", softcap=0.0, lens_q=[9, 11], lens_kv=[13, 6])]


def _case(i):
    kw = dict(CASES[i])
    if kw.get("rows") == "some":
        g = torch.Generator().manual_seed(i)
        lo = torch.randint(0, 9, (2, 11), generator=g)
        hi = lo + torch.randint(-1, 8, (2, 11), generator=g)
        kw["rows"] = torch.stack((lo, hi), -1).tolist()
    return Case(2, 2, 1, 11, 13, 8, 8, io=torch.float64, seed=i, gain=2.0, **kw)


def _loss(case):
    """sum(O * dO) by autograd-friendly float64 torch, written apart from Case."""
    total = 0.0
    for b in range(case.B):
        see, diag = visible(case.Sq, case.Skv, *case._lens(b), rows=None if case.rows is None else case.rows[b],
                            **case.mask)
        for h in range(case.Hq):
            x = case.q[b, h] @ case.k[b, 0].T * case.scale
            if case.softcap:
                x = case.softcap * torch.tanh(x / case.softcap)
            if case.slopes is not None:
                x = x - case.slopes[h].double() * (torch.arange(case.Sq)[:, None] + diag - torch.arange(case.Skv)).abs()
            w = torch.where(see, torch.exp(x), 0.0)
            z = w.sum(1, keepdim=True)
            o = (w / torch.where(z == 0, 1.0, z)) @ case.v[b, 0]
            total = total + (o * case.do[b, h]).sum()
    return total


@pytest.mark.parametrize("i", range(len(CASES)))
def test_reference_against_autograd_and_differences(i):
    case = _case(i)
    o, lse, _, _ = case.forward()
    (dq, dk, dv), _ = case.backward(o, lse)
    for t in (case.q, case.k, case.v):
        t.requires_grad_(True)
    loss = _loss(case)
    assert math.isclose(loss.item(), (o * case.do).sum().item(), rel_tol=1e-12, abs_tol=1e-12)
    grads = torch.autograd.grad(loss, (case.q, case.k, case.v))
    for a, g in zip((dq, dk, dv), grads):
        assert (a - g).abs().max() <= 1e-12 * (1 + g.abs().max())
    g = torch.Generator().manual_seed(99 + i)
    with torch.no_grad():
        for name, a in (("q", dq), ("k", dk), ("v", dv)):
            t = getattr(case, name)
            d = torch.randn(t.shape, generator=g, dtype=torch.float64)
            h = 1e-5
            setattr(case, name, t + h * d)
            up = _loss(case)
            setattr(case, name, t - h * d)
            down = _loss(case)
            setattr(case, name, t)
            # central differences: h^2 times the third derivative (a few units here) and
            # the loss's rounding (1e-14) over h
            assert abs((up - down) / (2 * h) - (a * d).sum()) <= 1e-7 * (1 + (a * d).abs().sum())


@pytest.mark.parametrize("S,gain", [(77, 1.0), (333, 3.0), (700, 1.0)])
def test_the_fp16_bound_sees_one_rounding(S, gain):
    """Weights rounded once to fp16 are within it; weights rounded to bf16, or a unit off, are not."""
    case = Case(1, 1, 1, S, S, 64, 64, io=torch.float16, seed=43, gain=gain, softcap=20.0, causal=True)
    ro, _, bo, _ = case.forward()
    bound = fp16_bound(case, bo)[0, 0]
    q, k, v, x, f, e = case.head(0, 0)
    p = torch.exp(x - x.amax(1, keepdim=True))
    for weight, fits in ((p.half().double(), True), (p.bfloat16().double(), False), (p.half().double() * (1 + 2.0 ** -9), False)):
        o = (weight @ v / p.sum(1, keepdim=True)).half().double()
        assert bool(((o - ro[0, 0]).abs() <= bound).all()) == fits
