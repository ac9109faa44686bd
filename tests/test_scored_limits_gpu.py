"""Attention with modified scores at the ends of its ranges, on the GPU against the
64-bit reference: calls in which no row sees a key, caps far above the usual scores, padded
rows of any finite values, fp16 weights. Bounds: scored_reference."""
import math

import pytest
import torch

from scored_reference import G23, Case, assert_within
from test_scored_gpu import _kw, _plan, _sdpa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("how", ["plan", "plan and cap", "lengths", "lengths and cap"])
@pytest.mark.parametrize("deterministic", [False, True])
def test_a_call_in_which_no_row_sees_a_key(deterministic, how, dims):
    """Zero gradients from every kernel of the chain, whatever the workspace held: the last one
    must not run ahead of the one that clears what it reads, although the one between them
    has nothing to compute. (The workspace's bytes are 3e38 as fp32, and a ticket past every unit.)"""
    if deterministic and "plan" in how and dims[0] == 64:
        pytest.skip("the ordered relay takes no plan")
    sdpa = _sdpa()
    B, Hq, Hkv, Sq, Skv = 2, 4, 2, 4000, 1000
    g = torch.Generator(device="cuda").manual_seed(44)
    q, k, v, do = (torch.randn(B, H, S, D, generator=g, device="cuda").bfloat16()
                   for H, S, D in ((Hq, Sq, dims[0]), (Hkv, Skv, dims[0]), (Hkv, Skv, dims[1]), (Hq, Sq, dims[1])))
    kw = dict(softcap=20.0 if "cap" in how else 0.0)
    if "plan" in how:
        nothing = torch.zeros(B, Sq, dtype=torch.int32, device="cuda")
        kw["mask_plan"] = sdpa.mask_plan(B, Sq, Skv, row_lo=nothing, row_hi=nothing)
    else:
        kw["seq_q_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    o, lse = sdpa.sdpa_fwd(q, k, v, **kw)
    assert (o == 0).all() and (lse == -math.inf).all()
    room = torch.empty(sdpa.workspace_size(B, Hq, Hkv, Sq, Skv, *dims, deterministic, padded=True, scored=True),
                       dtype=torch.uint8, device="cuda")
    for _ in range(20):
        room.fill_(0x7F)
        outs = {n: torch.full_like(t, math.nan) for n, t in (("dq", q), ("dk", k), ("dv", v))}
        got = sdpa.sdpa_bwd(q, k, v, o, do, lse, deterministic=deterministic, workspace=room, **outs, **kw)
        for name, t in zip(("dq", "dk", "dv"), got):
            assert (t == 0).all(), name
    sdpa.check_device_status()


class OneColumn(Case):
    """Queries and keys with one column that is not 0, keys of ones: a score is one exact
    product, so that scores of any size keep a small bound. What is left of a score's error
    is relative: scale / cap, the cap in log2 units and their products round to fp32 (5 roundings),
    the tanh is off by 3.1e-7 with its own roundings (5 more), and the exponent's argument rounds once: 11
    half units of fp32 of the largest capped score, taken as 6 units."""

    def __init__(self, *a, share, **kw):
        super().__init__(*a, **kw)
        y = share * self.softcap / self.scale  # q . k: scale * q . k is `share` caps
        self.q = torch.zeros_like(self.q)
        self.q[..., 0] = (y * torch.linspace(-1.0, 1.0, self.Sq)).to(self.io)
        self.k = torch.zeros_like(self.k)
        self.k[..., 0] = 1.0

    def head(self, b, h):
        q, k, v, x, f, _ = super().head(b, h)
        return q, k, v, x, f, 6 * G23 * x[torch.isfinite(x)].abs().max().item()


@pytest.mark.parametrize("dims", [(64, 64), (80, 80), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("share", [0.2, 0.64, 2.5])
@pytest.mark.parametrize("softcap,io", [(50.0, torch.bfloat16), (900.0, torch.float16), (2e3, torch.float16), (5e3, torch.bfloat16),
                                        (1e4, torch.bfloat16), (1e6, torch.bfloat16)])
def test_scores_near_a_large_cap(softcap, io, share, dims):
    """Scores up to 0.2, 0.64 (under the polynomial's bound) and 2.5 caps: LSE holds the capped score
    itself, and the backward gets the exact one."""
    if io == torch.float16 and share * softcap * 16 > 6e4:
        pytest.skip("no such fp16 score")
    case = OneColumn(1, 2, 1, 150, 391, *dims, io=io, seed=40, softcap=softcap, share=share)
    sdpa = _sdpa()
    q, k, v, do = (t.cuda() for t in (case.q, case.k, case.v, case.do))
    o, lse = sdpa.sdpa_fwd(q, k, v, softcap=softcap)
    ro, rl, bo, bl = case.forward()
    assert_within("o", o, ro, bo)
    assert_within("lse", lse, rl, bl)
    o, lse = ro.to(io), rl.float()
    ref, bounds = case.backward(o, lse)
    for det in (False, True):
        got = sdpa.sdpa_bwd(q, k, v, o.cuda(), do, lse.cuda(), softcap=softcap, deterministic=det)
        for name, g, r, b in zip(("dq", "dk", "dv"), got, ref, bounds):
            assert_within(f"{name} (deterministic={det})", g, r, b)


@pytest.mark.parametrize("mods", ["cap", "slopes", "both", "rows"])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("L", [1, 100, 128])
def test_padded_query_rows_may_be_huge(L, dims, mods):
    """Query rows past the length carry the io type's largest values in Q and dO: their
    scores and dP overflow to infinities and NaN, and must not reach any gradient."""
    S, Skv = 200, 140
    case = Case(1, 4, 2, S, Skv, *dims, seed=41, softcap=8.0 if mods in ("cap", "both") else 0.0,
                slopes=[0.1, 1.0, 0.0, 0.02] if mods in ("slopes", "both") else None,
                rows=[[(0, Skv)] * S] if mods == "rows" else None)
    most = torch.finfo(case.io).max
    sign = torch.where(torch.rand(S - L, 1, generator=torch.Generator().manual_seed(2)) < 0.5, -most, most)
    case.q[:, :, L:], case.do[:, :, L:] = sign.to(case.io), sign.flip(0).to(case.io)
    case.lens_q = [L]
    sdpa = _sdpa()
    q, k, v, do = (t.cuda() for t in (case.q, case.k, case.v, case.do))
    kw = _kw(case, _plan(case))
    o, lse = sdpa.sdpa_fwd(q, k, v, **kw)
    assert (o[:, :, L:] == 0).all() and (lse[:, :, L:] == -math.inf).all()
    got = {det: sdpa.sdpa_bwd(q, k, v, o, do, lse, deterministic=det, **kw)
           for det in ((False, True) if mods != "rows" or dims[0] >= 128 else (False,))}
    case.q, case.do, case.Sq, case.lens_q = case.q[:, :, :L], case.do[:, :, :L], L, None
    case.rows = None
    ro, rl, bo, bl = case.forward()
    assert_within("o", o[:, :, :L], ro, bo)
    assert_within("lse", lse[:, :, :L], rl, bl)
    ref, bounds = case.backward(o[:, :, :L].cpu(), lse[:, :, :L].cpu())
    for det, (dq, dk, dv) in got.items():
        assert (dq[:, :, L:] == 0).all()
        for name, g, r, b in zip(("dq", "dk", "dv"), (dq[:, :, :L], dk, dv), ref, bounds):
            assert_within(f"{name} (deterministic={det})", g, r, b)


def fp16_bound(case, bo):
    """Case.forward's bound of O with one rounding of each fp16 weight: an absolute part of 2^-25
    for a weight below 2^-14 of the row's reference. The reference is a score of the row (or its
    sink), whose weight is 1 in the sum that divides O, so the part reaches O times 1 at most.
    (Case.forward allows 256 times that part, several times everything else at a few hundred keys.)"""
    size = case.v.double().abs().sum(2).repeat_interleave(case.Hq // case.Hkv, 1)
    return bo - 255 * 2.0 ** -25 * size[:, :, None]


@pytest.mark.parametrize("dims", [(64, 64), (80, 80), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("mods", [dict(softcap=20.0), dict(slopes=[0.5, 0.02, 0.0]), dict(softcap=6.0, slopes=[0.5, 0.02, 0.0]),
                                  dict(rows=True), dict(rows=True, softcap=30.0, sink=True)])
@pytest.mark.parametrize("S,gain", [(77, 1.0), (333, 3.0), (700, 1.0)])
def test_fp16_outputs_by_their_own_roundings(S, gain, mods, dims):
    mods = dict(mods)
    if mods.pop("rows", False):
        mods["rows"] = [[(max(0, i // 90 * 90 - 7), min(S, i + 40)) for i in range(S)]] * 2
    else:
        mods["causal"] = True
    case = Case(2, 3, 1, S, S, *dims, io=torch.float16, seed=43, gain=gain, **mods)
    o, lse = _sdpa().sdpa_fwd(case.q.cuda(), case.k.cuda(), case.v.cuda(), **_kw(case, _plan(case)))
    ro, rl, bo, bl = case.forward()
    assert_within("o", o, ro, fp16_bound(case, bo))
    assert_within("lse", lse, rl, bl)
