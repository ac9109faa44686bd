"""Tensors that a call makes for a stream given to it (GPU): their memory must not be what
work queued elsewhere still uses, nor be given away while the call's own work uses it. Shown by
the addresses that torch's allocator hands out, with the streams held up, so that nothing here
depends on a race."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, HQ, HKV, S, D = 1, 4, 2, 512, 64
HOLD = 200_000_000  # clock cycles, about 0.1 s


def _sdpa():
    import attention_backward_sdpa_gb300 as pkg
    return pkg


def _inputs():
    q, o, do = (torch.randn(B, HQ, S, D, device="cuda").bfloat16() for _ in range(3))
    k, v = (torch.randn(B, HKV, S, D, device="cuda").bfloat16() for _ in range(2))
    return q, k, v, o, do, torch.zeros(B, HQ, S, device="cuda")


def _calls():
    """Name -> (call on a stream, returning the tensors that it made)."""
    sdpa = _sdpa()
    q, k, v, o, do, lse = _inputs()
    freq = sdpa.rope_inv_freq(D)
    ids = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    bias, sink = torch.zeros(1, HQ, S, S, device="cuda"), torch.zeros(HQ, device="cuda")
    wide = [torch.randn(B, H, S, 128, device="cuda").bfloat16() for H in (HQ, HKV, HKV, HQ, HQ)]
    return {
        "mask_plan": lambda s: (sdpa.mask_plan(B, S, S, doc_ids=ids, causal=True, stream=s).buffer,),
        "rope_fwd": lambda s: sdpa.rope_fwd(q, k, freq, stream=s),
        "rope_bwd": lambda s: sdpa.rope_bwd(q, k, freq, stream=s),
        "sdpa_fwd": lambda s: sdpa.sdpa_fwd(q, k, v, stream=s),
        "sdpa_fwd capped": lambda s: sdpa.sdpa_fwd(q, k, v, softcap=9.0, stream=s),
        "sdpa_bwd": lambda s: sdpa.sdpa_bwd(q, k, v, o, do, lse, stream=s),
        "sdpa_bwd capped": lambda s: sdpa.sdpa_bwd(q, k, v, o, do, lse, softcap=9.0, sink=sink, stream=s),
        "sdpa_bwd biased": lambda s: sdpa.sdpa_bwd(q, k, v, o, do, lse, bias=bias, stream=s),
        "nvfp4_fake_quant": lambda s: (sdpa.nvfp4_fake_quant(q, stream=s),),
        "sdpa_bwd_nvfp4_qat": lambda s: sdpa.sdpa_bwd_nvfp4_qat(*wide, lse, stream=s),
    }


NAMES = ["mask_plan", "rope_fwd", "rope_bwd", "sdpa_fwd", "sdpa_fwd capped", "sdpa_bwd", "sdpa_bwd capped",
         "sdpa_bwd biased", "nvfp4_fake_quant", "sdpa_bwd_nvfp4_qat"]


def _blocks(tensors):
    return {t.data_ptr() for t in tensors}


@pytest.mark.parametrize("name", NAMES)
def test_outputs_do_not_take_what_the_current_stream_still_uses(name):
    call, side = _calls()[name], torch.cuda.Stream()
    sizes = [t.untyped_storage().nbytes() for t in call(side)]  # (and the kernels are loaded)
    torch.cuda.synchronize()
    held = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(HOLD)
    for t in held:
        t.fill_(1)  # queued behind the sleep
    before = _blocks(held)
    del held, t
    assert not before & _blocks(call(side))
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_outputs_stay_until_both_streams_are_done_with_them(name):
    """Made on a stream, read on the current one, dropped while either still works: neither stream
    gets the memory for anything else before."""
    call, side = _calls()[name], torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    for busy in ("current", "side"):
        if busy == "side":
            with torch.cuda.stream(side):
                torch.cuda._sleep(HOLD)
        made = call(side)
        if busy == "current":
            torch.cuda._sleep(HOLD)
            torch.cuda.current_stream().wait_stream(side)
        else:
            assert not side.query()
        sizes, before = [t.untyped_storage().nbytes() for t in made], _blocks(made)
        del made
        other = torch.cuda.current_stream() if busy == "side" else side
        with torch.cuda.stream(other):
            assert not before & _blocks([torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes])
        torch.cuda.synchronize()


def test_a_plan_that_is_dropped_while_another_stream_reads_it():
    """Made on the current stream, read by calls on another one that is held up."""
    sdpa = _sdpa()
    q, k, v, o, do, lse = _inputs()
    ids = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    outs = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    for call in (lambda p: sdpa.sdpa_fwd(q, k, v, o=o, lse=lse, mask_plan=p, stream=side),
                 lambda p: sdpa.sdpa_bwd(q, k, v, o, do, lse, mask_plan=p, stream=side, **outs)):
        plan = sdpa.mask_plan(B, S, S, doc_ids=ids, causal=True)
        call(plan)  # (the kernels are loaded)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD)
        call(plan)
        size, before = plan.buffer.numel(), plan.buffer.data_ptr()
        del plan
        assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != before
        torch.cuda.synchronize()
    # ... and where the stream is the current one at the call
    plan = sdpa.mask_plan(B, S, S, doc_ids=ids, causal=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
        sdpa.sdpa_fwd(q, k, v, o=o, lse=lse, mask_plan=plan)
    size, before = plan.buffer.numel(), plan.buffer.data_ptr()
    del plan
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != before
    torch.cuda.synchronize()


def test_a_captured_step_on_a_given_stream():
    """The same calls inside a graph, on a stream that was forked from the capturing one."""
    sdpa = _sdpa()
    q, k, v, _, do, _ = _inputs()
    freq = sdpa.rope_inv_freq(D)
    ids = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    ids[:, 200:] = 1
    side = torch.cuda.Stream()

    def step(stream):
        plan = sdpa.mask_plan(B, S, S, doc_ids=ids, causal=True, stream=stream)
        a, b = sdpa.rope_fwd(q, k, freq, stream=stream)
        o, lse = sdpa.sdpa_fwd(a, b, v, softcap=9.0, mask_plan=plan, stream=stream)
        room = torch.empty(sdpa.workspace_size(B, HQ, HKV, S, S, D, D, scored=True), dtype=torch.uint8, device="cuda")
        return (o, lse) + sdpa.sdpa_bwd(a, b, v, o, do, lse, softcap=9.0, mask_plan=plan, workspace=room, stream=stream)

    want = step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got[:2], want[:2]):
            assert torch.equal(x, y)
        for x, y in zip(got[2:], want[2:]):  # (dQ's reduction adds in any order)
            assert (x.float() - y.float()).abs().max() <= 2.0 ** -6 * y.float().abs().max()
