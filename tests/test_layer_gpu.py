"""The operators as a layer's training step uses them: rotary embedding of the
projections, attention with capped, biased scores over packed documents, its gradient,
and the rotation's gradient back into the projections' layout. Each stage is compared
with the 64-bit reference of that stage on the inputs that it got; the whole step's
gradients with 64-bit autograd of the whole step."""
import pytest
import torch

from scored_reference import Case, assert_within, doc_ranges

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rot,interleaved,io", [(64, 64, False, torch.bfloat16), (128, 64, True, torch.float16),
                                                  (256, 256, False, torch.bfloat16)])
def test_training_step(D, rot, interleaved, io):
    import attention_backward_sdpa_gb300 as sdpa
    B, S, Hq, Hkv, cap = 2, 190, 4, 2, 12.0
    ids = torch.zeros(B, S, dtype=torch.int32)
    ids[0, 70:], ids[1, 33:], ids[1, 128:] = 1, 1, 2
    pos = torch.arange(S).expand(B, S).clone()
    for b in range(B):
        for d in range(3):
            at = (ids[b] == d).nonzero().flatten()
            if at.numel():
                pos[b, at] -= at[0]
    pos = pos.to(torch.int32)
    slopes = [0.25, 0.05, 0.0, 0.5]
    case = Case(B, Hq, Hkv, S, S, D, D, io=io, seed=5, softcap=cap, slopes=slopes,
                rows=doc_ranges(ids.tolist(), None, True, S))
    # The projections' outputs, (B, S, H, D).
    xq, xk = (t.transpose(1, 2).contiguous() for t in (case.q, case.k))
    f = sdpa.rope_inv_freq(rot)
    kw = dict(positions=pos.cuda(), interleaved=interleaved, mult=1.1)
    q, k = sdpa.rope_fwd(xq.cuda().transpose(1, 2), xk.cuda().transpose(1, 2), f, **kw)
    plan = sdpa.mask_plan(B, S, S, doc_ids=ids.cuda(), causal=True)
    mods = dict(softcap=cap, alibi_slopes=case.slopes.cuda(), mask_plan=plan)
    v, do = case.v.cuda(), case.do.cuda()
    o, lse = sdpa.sdpa_fwd(q, k, v, **mods)
    dq, dk, dv = sdpa.sdpa_bwd(q, k, v, o, do, lse, **mods)
    gq, gk = (torch.empty_like(t, device="cuda") for t in (xq, xk))
    sdpa.rope_bwd(dq, dk, f, q_out=gq.transpose(1, 2), k_out=gk.transpose(1, 2), **kw)
    sdpa.check_device_status()

    # Stage by stage.
    case.q, case.k = q.cpu(), k.cpu()
    ro, rl, bo, bl = case.forward()
    assert_within("o", o, ro, bo)
    assert_within("lse", lse, rl, bl)
    ref, bounds = case.backward(o.cpu(), lse.cpu())
    for name, got, r, bound in zip(("dq", "dk", "dv"), (dq, dk, dv), ref, bounds):
        assert_within(name, got, r, bound)

    # The whole step in 64 bits by autograd: the roundings in between (q, k, O, dQ, dK to
    # the io type) perturb the scores by u |x| each way and the rest relatively, a few u
    # of the gradients' size. In the 2-norm: q and k rounded shift every score by a
    # random part of sqrt(2) u |score|, |score| up to about 1.1^2 * 12, so P and dS by up
    # to 15 sqrt(2) u relative; O, dS, dQ, dK and the output add a u each: 26 u.
    x64, k64, v64 = (t.double().requires_grad_(True) for t in (xq, xk, case.v))
    angle = pos.double()[..., None] * f.cpu()
    c, s = torch.cos(angle)[:, :, None] * 1.1, torch.sin(angle)[:, :, None] * 1.1

    def turn(x):
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = (a * c - b * s, b * c + a * s)
        y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
        return torch.cat((y, x[..., rot:]), -1).transpose(1, 2)

    G = Hq // Hkv
    y = turn(x64) @ turn(k64).repeat_interleave(G, 1).transpose(2, 3) * case.scale
    i = torch.arange(S)
    y = cap * torch.tanh(y / cap) - case.slopes.double().view(1, -1, 1, 1) * (i[:, None] - i).abs()
    r = torch.tensor(case.rows)
    see = (i >= r[..., :1]) & (i < r[..., 1:])
    p = torch.softmax(y.masked_fill(~see[:, None], float("-inf")), -1)
    loss = ((p @ v64.repeat_interleave(G, 1)) * case.do.double()).sum()
    u = torch.finfo(io).eps / 2
    for name, got, want in zip(("dq", "dk", "dv"), (gq, gk, dv), torch.autograd.grad(loss, (x64, k64, v64))):
        err = (got.cpu().double() - want).norm() / want.norm()
        assert err <= 26 * u, f"{name}: {err:.3e}"
