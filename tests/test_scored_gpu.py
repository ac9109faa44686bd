"""Attention with modified scores (softcap, distance slopes, row ranges) on the GPU
against the 64-bit reference, forward and backward, at the sizes and masks where
it can go wrong. Bounds: scored_reference."""
import math

import pytest
import torch

from scored_reference import Case, assert_within, doc_ranges

pytestmark = pytest.mark.gpu


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def _ids(B, S, cuts):
    return [[sum(i >= c for c in cuts[b % len(cuts)]) for i in range(S)] for b in range(B)]


def _dev(x, dtype=None):
    return None if x is None else (x if isinstance(x, torch.Tensor) else torch.tensor(x, dtype=dtype)).cuda()


def _plan(case):
    """A plan of the case's row ranges through the general form."""
    if case.rows is None:
        return None
    r = torch.tensor(case.rows, dtype=torch.int32)
    return _sdpa().mask_plan(case.B, case.Sq, case.Skv, row_lo=r[..., 0].contiguous().cuda(),
                             row_hi=r[..., 1].contiguous().cuda())


def _kw(case, plan):
    return dict(softcap=case.softcap, alibi_slopes=_dev(case.slopes), mask_plan=plan,
                seq_q_lens=_dev(case.lens_q, torch.int32), seq_kv_lens=_dev(case.lens_kv, torch.int32),
                sink=_dev(case.sink), **case.mask)


def _check(case, plan=None, deterministic=(False,)):
    sdpa = _sdpa()
    plan = _plan(case) if plan is None else plan
    kw = _kw(case, plan)
    q, k, v, do = (t.cuda() for t in (case.q, case.k, case.v, case.do))
    o = torch.full((case.B, case.Hq, case.Sq, case.Dv), math.nan, dtype=case.io, device="cuda")
    lse = torch.full((case.B, case.Hq, case.Sq), math.nan, device="cuda")
    sdpa.sdpa_fwd(q, k, v, o=o, lse=lse, **kw)
    sdpa.check_device_status()
    ro, rl, bo, bl = case.forward()
    assert_within("o", o, ro, bo)
    assert_within("lse", lse, rl, bl)
    ref, bounds = case.backward(o.cpu(), lse.cpu())
    for det in deterministic:
        outs = {n: torch.full_like(t, math.nan) for n, t in (("dq", q), ("dk", k), ("dv", v))}
        got = sdpa.sdpa_bwd(q, k, v, o, do, lse, deterministic=det, **outs, **kw)
        sdpa.check_device_status()
        for name, g, r, b in zip(("dq", "dk", "dv"), got, ref, bounds):
            assert_within(f"{name} (deterministic={det})", g, r, b)
    return o, lse


DIMS = [(64, 64), (128, 128), (8, 8), (80, 80), (192, 128), (256, 256)]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("mods", ["cap", "slopes", "both"])
def test_cap_and_slopes(dims, io, mods):
    case = Case(2, 4, 2, 150, 150, *dims, io=io, seed=1, gain=2.0, causal=True,
                softcap=20.0 if mods != "slopes" else 0.0, slopes=[0.5, 0.25, 0.0, -0.01] if mods != "cap" else None)
    _check(case, deterministic=(False, True))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dims", DIMS)
def test_documents_with_prefix(dims, io):
    B, S = 2, 333
    ids = _ids(B, S, [[1, 40, 128, 129, 200], [64, 300]])
    pre = [3, 70]
    case = Case(B, 4, 2, S, S, *dims, io=io, seed=2, rows=doc_ranges(ids, pre, True, S), softcap=30.0)
    plan = _sdpa().mask_plan(B, S, S, doc_ids=_dev(ids, torch.int32), prefix_lens=_dev(pre, torch.int32), causal=True)
    _check(case, plan, deterministic=(False, True) if dims[0] in (128, 192, 256) else (False,))


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (256, 256)])
@pytest.mark.parametrize("case_id", range(6))
def test_row_ranges_of_any_kind(dims, case_id):
    """Rows without keys, ranges that jump back and forth, whole empty batch rows, single keys."""
    B, Sq, Skv = 2, 200, 391
    g = torch.Generator().manual_seed(100 + case_id)
    lo = torch.randint(-5, Skv + 5, (B, Sq), generator=g)
    hi = lo + torch.randint(-20, 150, (B, Sq), generator=g)
    if case_id == 1:
        lo[0], hi[0] = 0, 0                   # no row of a batch row sees a key
    if case_id == 2:
        lo[:, :], hi[:, :] = 0, Skv           # everything
    if case_id == 3:
        lo[:], hi[:] = 390, 391               # the last key alone
    if case_id == 4:
        lo[:, 64:128], hi[:, 64:128] = 7, 7   # one query tile without a key
        lo[:, ::2], hi[:, ::2] = 0, 1
    if case_id == 5:                          # far apart ranges in neighbouring rows
        lo[:, ::2], hi[:, ::2] = 0, 3
        lo[:, 1::2], hi[:, 1::2] = 380, 400
    rows = torch.stack((lo, hi), -1).tolist()
    case = Case(B, 2, 1, Sq, Skv, *dims, seed=3 + case_id, rows=rows, softcap=15.0 if case_id % 2 else 0.0)
    _check(case, deterministic=(False, True) if dims[0] >= 128 else (False,))


@pytest.mark.parametrize("Sq,Skv", [(1, 1), (1, 300), (65, 1), (64, 128), (129, 257), (2, 4097)])
def test_sizes(Sq, Skv):
    rows = [[(max(0, j - 40), min(Skv, j + 3)) for j in range(Sq)]] * 2
    case = Case(2, 3, 3, Sq, Skv, 64, 64, seed=4, rows=rows, softcap=10.0, slopes=[1.0, 0.1, 3.0])
    _check(case)
    _check(Case(2, 3, 1, Sq, Skv, 128, 128, seed=5, softcap=50.0, gain=4.0, causal=True, bottom_right=True),
           deterministic=(False, True))


@pytest.mark.parametrize("mask", [dict(causal=True, bottom_right=True), dict(causal=True, window_left=37),
                                  dict(causal=True, window_right=9), dict(window_left=20, bottom_right=True),
                                  dict()])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
def test_with_the_other_masks(mask, dims):
    """Ranges, cap and slopes together with causal, window and lengths (one batch row empty), and a sink."""
    B, Sq, Skv = 3, 180, 260
    ids = _ids(B, Skv, [[100, 131], [5], []])
    rows = [r[:Sq] for r in doc_ranges(ids, None, False, Skv)]
    case = Case(B, 4, 2, Sq, Skv, *dims, seed=6, rows=rows, softcap=25.0, slopes=[0.3, 0.05, 0.0, 0.7],
                lens_q=[180, 77, 0], lens_kv=[260, 200, 131], sink=True, **mask)
    _check(case, deterministic=(False, True) if dims[0] >= 128 else (False,))


@pytest.mark.parametrize("softcap,gain", [(0.25, 30.0), (5.0, 60.0), (50.0, 40.0), (1e4, 1.0), (1e30, 3.0), (1e-3, 1.0)])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128)])
def test_caps_far_from_the_scores(softcap, gain, dims):
    """Scores far above the cap (saturated), mixed ones, and a cap far above every score."""
    _check(Case(1, 2, 2, 140, 140, *dims, seed=7, softcap=softcap, gain=gain, causal=True))


def test_masked_scores_may_be_huge():
    """Keys that the ranges mask carry the io type's largest values: their scores
    overflow the cap's argument or the bias, and must not reach any output."""
    S = 160
    case = Case(1, 2, 2, S, S, 64, 64, io=torch.bfloat16, seed=8, softcap=5.0, slopes=[0.1, 2.0],
                rows=[[(0, 100)] * S])
    big = case.k.clone()
    big[:, :, 100:] = torch.finfo(torch.bfloat16).max
    case.k = big
    sdpa = _sdpa()
    plan = _plan(case)
    q, k, v, do = (t.cuda() for t in (case.q, case.k, case.v, case.do))
    o, lse = sdpa.sdpa_fwd(q, k, v, softcap=5.0, alibi_slopes=_dev(case.slopes), mask_plan=plan)
    got = sdpa.sdpa_bwd(q, k, v, o, do, lse, softcap=5.0, alibi_slopes=_dev(case.slopes), mask_plan=plan)
    case.k = case.k[:, :, :100]
    case.v, case.Skv, case.rows = case.v[:, :, :100], 100, None
    ro, rl, bo, bl = case.forward()
    assert_within("o", o, ro, bo)
    assert_within("lse", lse, rl, bl)
    ref, bounds = case.backward(o.cpu(), lse.cpu())
    assert_within("dq", got[0], ref[0], bounds[0])
    for g, r, b in zip(got[1:], ref[1:], bounds[1:]):
        assert_within("dk, dv", g[:, :, :100], r, b)
        assert (g[:, :, 100:] == 0).all()


def test_a_plan_that_masks_nothing():
    """It gives the plain call's results: dQ bit for bit (the same operations in the same
    order); O and LSE, whose exponents and sums are formed in another order, and dK and
    dV, whose group sums are rounded once instead of once per head as well, within the
    bounds that they keep to the exact result."""
    sdpa = _sdpa()
    c = Case(2, 4, 2, 200, 200, 128, 128, seed=9, causal=True)
    q, k, v, do = (t.cuda() for t in (c.q, c.k, c.v, c.do))
    everything = torch.zeros(2, 200, dtype=torch.int32, device="cuda")
    plan = sdpa.mask_plan(2, 200, 200, row_lo=everything, row_hi=everything + 200)
    a, b = sdpa.sdpa_fwd(q, k, v, causal=True), sdpa.sdpa_fwd(q, k, v, causal=True, mask_plan=plan)
    ro, rl, bo, bl = c.forward()
    for o, lse in (a, b):
        assert_within("o", o, ro, bo)
        assert_within("lse", lse, rl, bl)
    x = sdpa.sdpa_bwd(q, k, v, a[0], do, a[1], causal=True, deterministic=True)
    y = sdpa.sdpa_bwd(q, k, v, a[0], do, a[1], causal=True, deterministic=True, mask_plan=plan)
    assert torch.equal(x[0], y[0])
    ref, bounds = c.backward(a[0].cpu(), a[1].cpu())
    for name, g, r, bound in zip(("dq", "dk", "dv"), y, ref, bounds):
        assert_within(name, g, r, bound)


@pytest.mark.parametrize("B,S", [(1, 1), (2, 63), (3, 1025), (2, 5000)])
@pytest.mark.parametrize("prefix", [None, "batch", "row"])
def test_plan_ranges(B, S, prefix):
    """The ranges and both summaries of a plan, from random ids that come back (runs are
    documents), against the definition."""
    sdpa = _sdpa()
    g = torch.Generator().manual_seed(S)
    ids = torch.repeat_interleave(torch.randint(0, 3, (B, S), generator=g), torch.randint(1, 200, (S,), generator=g),
                                  dim=1)[:, :S].contiguous().to(torch.int32)
    pre = None
    if prefix == "batch":
        pre = torch.randint(-3, 90, (B,), generator=g, dtype=torch.int32)
    elif prefix == "row":
        pre = torch.randint(-3, 2 * S, (B, S), generator=g, dtype=torch.int32)
    plan = sdpa.mask_plan(B, S, S, doc_ids=ids.cuda(), prefix_lens=_dev(pre), causal=True)
    n_qt, n_kt = -(-S // 64), -(-S // 128)
    words = plan.buffer.cpu().view(torch.int32)
    ranges = words[: B * n_qt * 64 * 2].view(B, n_qt * 64, 2)
    rows = torch.zeros(B, S, 2, dtype=torch.int32)
    edge = torch.ones(B, S + 1, dtype=torch.bool)
    edge[:, 1:S] = ids[:, 1:] != ids[:, :-1]
    pos = torch.arange(S + 1)
    for b in range(B):
        starts = pos[edge[b]]
        lo = starts[torch.searchsorted(starts, pos[:S], right=True) - 1]
        hi = starts[torch.searchsorted(starts, pos[:S], right=True)]
        p = torch.zeros(S, dtype=torch.long) if pre is None else pre[b].long().expand(S).clamp(min=0)
        hi = torch.minimum(hi, torch.maximum(pos[:S] + 1, lo + p))
        rows[b, :, 0], rows[b, :, 1] = lo, hi
    assert torch.equal(ranges[:, :S], rows)
    assert (ranges[:, S:] == 0).all()
    up = lambda x: (x + 63) // 64 * 64  # noqa: E731  (256 bytes)
    at = up(B * n_qt * 64 * 2)
    q_sum = words[at: at + B * n_qt * 4].view(B, n_qt, 4)
    at = up(at + B * n_qt * 4)
    k_sum = words[at: at + B * n_kt * 2].view(B, n_kt, 2)
    for b in range(B):
        for t in range(n_qt):
            r = rows[b, 64 * t: 64 * t + 64]
            assert q_sum[b, t].tolist() == [r[:, 0].min().item(), r[:, 1].max().item(), r[:, 0].max().item(),
                                            r[:, 1].min().item()]
        for t in range(n_kt):
            meet = [i for i in range(n_qt) if q_sum[b, i, 0] < 128 * (t + 1) and q_sum[b, i, 1] > 128 * t]
            assert k_sum[b, t].tolist() == ([meet[0], meet[-1]] if meet else [0, -1])
    # The rows that see each key, where they are neighbours (a prefix length that changes
    # within a document need not leave them so).
    at = up(at + B * n_kt * 2)
    k_rows = words[at: at + B * n_kt * 128 * 2].view(B, n_kt * 128, 2)
    k_exact = words[at + B * n_kt * 128 * 2:][:B]
    for b in range(B):
        lo, hi = rows[b, :, 0], rows[b, :, 1]
        up_to = bool((lo[1:] >= lo[:-1]).all() and (hi[1:] >= hi[:-1]).all())
        assert k_exact[b] == int(up_to)
        if up_to:
            for k in range(0, S, 1 if S < 2000 else 17):
                see = ((lo <= k) & (hi > k)).nonzero().flatten()
                assert see.numel() and k_rows[b, k].tolist() == [see[0].item(), see[-1].item()]
                assert see.numel() == see[-1] - see[0] + 1
    assert prefix == "row" or k_exact.all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_sink_gradient(D):
    """dsink = -sum exp(sink - LSE) delta over the live rows, within 2^-16 of the terms'
    magnitudes: an fp32 dot of D terms (D 2^-24 <= 2^-16), an exponent of about 20 in
    fp32 (20 2^-24 ln 2) and a sum of a few hundred terms."""
    sdpa = _sdpa()
    B, H, S = 2, 4, 130
    c = Case(B, H, 2, S, S, D, D, seed=12, softcap=9.0, slopes=[0.1, 0.0, 1.0, 0.02], sink=True, causal=True,
             lens_q=[130, 50], lens_kv=[130, 90])
    q, k, v, do = (t.cuda() for t in (c.q, c.k, c.v, c.do))
    kw = _kw(c, None)
    o, lse = sdpa.sdpa_fwd(q, k, v, **kw)
    dsink = sdpa.sdpa_bwd(q, k, v, o, do, lse, **kw)[3]
    delta = (do.double() * o.double()).sum(-1).cpu()
    term = torch.exp(c.sink.double()[None, :, None] - lse.double().cpu()) * delta
    size = torch.exp(c.sink.double()[None, :, None] - lse.double().cpu()) * (do.double() * o.double()).abs().sum(-1).cpu()
    for b in range(B):
        term[b, :, c.lens_q[b]:] = size[b, :, c.lens_q[b]:] = 0.0
    assert ((dsink.double().cpu() + term.sum((0, 2))).abs() <= 2.0 ** -16 * size.sum((0, 2))).all()


def test_repeated_calls_are_bitwise_equal():
    sdpa = _sdpa()
    B, S = 2, 700
    ids = _ids(B, S, [[100, 350], [512]])
    c = Case(B, 8, 2, S, S, 128, 128, seed=10, softcap=20.0, slopes=[0.1] * 8)
    plan = sdpa.mask_plan(B, S, S, doc_ids=_dev(ids, torch.int32), causal=True)
    q, k, v, do = (t.cuda() for t in (c.q, c.k, c.v, c.do))
    kw = dict(softcap=20.0, alibi_slopes=_dev(c.slopes), mask_plan=plan)
    o, lse = sdpa.sdpa_fwd(q, k, v, **kw)
    first = sdpa.sdpa_bwd(q, k, v, o, do, lse, deterministic=True, **kw)
    for _ in range(5):
        o2, lse2 = sdpa.sdpa_fwd(q, k, v, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(first, sdpa.sdpa_bwd(q, k, v, o, do, lse, deterministic=True, **kw)):
            assert torch.equal(a, b)


def test_two_streams_and_a_captured_step():
    """A step captured into a graph and replayed on new inputs while another stream
    runs the same calls eagerly; the plan is remade inside the graph."""
    sdpa = _sdpa()
    B, S, cap = 2, 450, 12.0
    cases = [Case(B, 4, 2, S, S, 128, 128, seed=20 + i, softcap=cap) for i in range(2)]
    ids = [_dev(_ids(B, S, [[90, 300], [17]]), torch.int32), _dev(_ids(B, S, [[200], [64, 65]]), torch.int32)]

    def step(q, k, v, do, ids):
        plan = sdpa.mask_plan(B, S, S, doc_ids=ids, causal=True)
        o, lse = sdpa.sdpa_fwd(q, k, v, softcap=cap, mask_plan=plan)
        return (o, lse) + sdpa.sdpa_bwd(q, k, v, o, do, lse, softcap=cap, mask_plan=plan, deterministic=True)

    inputs = [[t.cuda() for t in (c.q, c.k, c.v, c.do)] + [ids[i]] for i, c in enumerate(cases)]
    want = [step(*x) for x in inputs]
    torch.cuda.synchronize()
    fixed = [t.clone() for t in inputs[0]]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        out = step(*fixed)
    for i in (1, 0, 1):
        for a, b in zip(fixed, inputs[i]):
            a.copy_(b)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = step(*inputs[1 - i])
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)
        for a, b in zip(other, want[1 - i]):
            assert torch.equal(a, b)


def test_a_plan_may_be_written_again():
    sdpa = _sdpa()
    S = 200
    plan = sdpa.mask_plan(1, S, S, doc_ids=torch.zeros(1, S, dtype=torch.int32, device="cuda"), causal=True)
    before = plan.buffer.clone()
    ids = _dev(_ids(1, S, [[50]]), torch.int32)
    again = sdpa.mask_plan(1, S, S, doc_ids=ids, causal=True, plan=plan)
    assert again is plan and not torch.equal(before, plan.buffer)
    case = Case(1, 2, 2, S, S, 64, 64, seed=11, rows=doc_ranges(ids.tolist(), None, True, S))
    _check(case, plan)


def test_a_long_row_of_documents():
    """66,000 positions in one row: the documents' results are those of each document alone
    (its own rows, keys and distances), within the bounds of the document alone."""
    sdpa = _sdpa()
    S, H, D = 66000, 2, 64
    cuts = [0, 300, 40000, 65409, 65600, S]
    ids = torch.zeros(1, S, dtype=torch.int32)
    for c in cuts[1:-1]:
        ids[0, c:] += 1
    g = torch.Generator().manual_seed(31)
    q, k, v, do = (torch.randn(1, H, S, D, generator=g).bfloat16() for _ in range(4))
    slopes = [0.02, 0.3]
    plan = sdpa.mask_plan(1, S, S, doc_ids=ids.cuda(), causal=True)
    kw = dict(softcap=20.0, alibi_slopes=torch.tensor(slopes).cuda(), mask_plan=plan)
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = sdpa.sdpa_fwd(*dev[:3], **kw)
    got = sdpa.sdpa_bwd(*dev[:3], o, dev[3], lse, **kw)
    sdpa.check_device_status()
    for a, b in ((0, 300), (65409, 65600), (65600, S)):
        one = Case(1, H, H, b - a, b - a, D, D, softcap=20.0, slopes=slopes, causal=True)
        one.q, one.k, one.v, one.do = (t[:, :, a:b] for t in (q, k, v, do))
        ro, rl, bo, bl = one.forward()
        assert_within("o", o[:, :, a:b], ro, bo)
        assert_within("lse", lse[:, :, a:b], rl, bl)
        ref, bounds = one.backward(o[:, :, a:b].cpu(), lse[:, :, a:b].cpu())
        for name, t, r, bound in zip(("dq", "dk", "dv"), got, ref, bounds):
            assert_within(f"{name} of [{a}, {b})", t[:, :, a:b], r, bound)


@pytest.mark.parametrize("det", [False, True])
def test_a_workspace_of_the_exact_size_and_a_given_stream(det):
    sdpa = _sdpa()
    B, Hq, Hkv, S, D = 2, 6, 2, 200, 128
    c = Case(B, Hq, Hkv, S, S, D, D, seed=13, softcap=7.0, causal=True)
    q, k, v, do = (t.cuda() for t in (c.q, c.k, c.v, c.do))
    o, lse = sdpa.sdpa_fwd(q, k, v, softcap=7.0, causal=True)
    want = sdpa.sdpa_bwd(q, k, v, o, do, lse, softcap=7.0, causal=True, deterministic=True)
    n = sdpa.workspace_size(B, Hq, Hkv, S, S, D, D, det, causal=True, scored=True)
    room = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    got = sdpa.sdpa_bwd(q, k, v, o, do, lse, softcap=7.0, causal=True, deterministic=det, workspace=room[:n])
    assert (room[n:] == 0x5A).all()
    ref, bounds = c.backward(o.cpu(), lse.cpu())
    for g, w, r, b in zip(got, want, ref, bounds):
        assert_within("workspace", g, r, b)
        assert not det or torch.equal(g, w)
    with pytest.raises(sdpa.SdpaError):
        sdpa.sdpa_bwd(q, k, v, o, do, lse, softcap=7.0, causal=True, deterministic=det, workspace=room[:n - 256])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = sdpa.sdpa_fwd(q, k, v, softcap=7.0, causal=True, stream=side)
    other = sdpa.sdpa_bwd(q, k, v, o2, do, lse2, softcap=7.0, causal=True, deterministic=True, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(other, want):
        assert torch.equal(a, b)


def test_outputs_below_fp16_normals():
    """A sink that takes nearly all of the weight: outputs down to 1e-9, fp16 subnormals and zeros."""
    _check(Case(2, 3, 3, 1, 1, 80, 80, io=torch.float16, seed=2587, gain=15.0, sink=True, causal=True,
                bottom_right=True, window_left=0, slopes=[0.5, 0.0, 2.0]), deterministic=(False, True))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("softcap", [0.0, 30.0, 2.0])
@pytest.mark.parametrize("mask", [dict(), dict(bottom_right=True), dict(causal=True), dict(window_left=200)])
def test_slopes_on_both_sides_of_the_rows(mask, softcap, io):
    """Several key tiles before and behind every row; slopes of both signs, none, steep ones."""
    case = Case(1, 6, 2, 520, 700, 64, 64, io=io, seed=37, softcap=softcap,
                slopes=[0.002, 0.06, -0.003, 0.0, 1.5, 0.25], **mask)
    _check(case, deterministic=(False, True))
