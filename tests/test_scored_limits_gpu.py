"""Attention with modified scores at the ends of its ranges, on the GPU against the
64-bit reference: calls in which no row sees a key."""
import math

import pytest
import torch

from test_scored_gpu import _sdpa

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
