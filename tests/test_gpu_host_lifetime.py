"""Host tensors that the caller drops while a host-buffer call is in flight."""

import weakref

import pytest

from attn_inputs import BASE_SEED
from gpu_util import inputs, scale_f32
from test_gpu_host import host_bf16, run_device

pytestmark = pytest.mark.gpu

SHAPE = (1, 4, 768, 128)


def busy():
    """Keep the stream busy for some 50 ms, so that the copies behind it wait."""
    import torch
    torch.cuda._sleep(100_000_000)


def scribble(n):
    """What the caller does next: page-locked tensors of the same size, full of NaN."""
    import torch
    return [torch.full(SHAPE, float("nan"), dtype=torch.bfloat16).pin_memory() for _ in range(n)]


@pytest.mark.parametrize("own_stream", [False, True])
def test_inputs_that_are_dropped_at_once(own_stream):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, H, N, d = SHAPE
    x, _ = inputs(B, H, N, d, BASE_SEED + 1500)
    scale = scale_f32(d)
    stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
    buf = torch.empty(fa.fa_fwd_bwd_host_device_bytes(B, H, N, d), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(SHAPE, dtype=torch.bfloat16).pin_memory() for _ in range(5)]
    lse = [torch.empty((B, H, N)).pin_memory() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        busy()
    fa.fa_fwd_bwd_host(*(host_bf16(x[n], True) for n in ("q", "k", "v", "do")), outs[0], lse[0], *outs[1:4], False, scale, buf,
                       stream)
    held = scribble(6)
    fa.fa_fwd_host(*(host_bf16(x[n], True) for n in ("q", "k", "v")), outs[4], lse[1], False, scale, buf, stream)
    held += scribble(6)
    assert fa.fa_get_device_status(stream) == 0
    want = run_device(x, False, scale)
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), (outs[0], lse[0], *outs[1:4]), want):
        assert torch.equal(a, b), name
    assert torch.equal(outs[4], want[0]) and torch.equal(lse[1], want[1])
    assert all(t.isnan().all() for t in held)


def test_outputs_that_are_dropped_at_once_write_nowhere_else():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, H, N, d = SHAPE
    x, _ = inputs(B, H, N, d, BASE_SEED + 1501)
    ins = [host_bf16(x[n], True) for n in ("q", "k", "v")]
    buf = torch.empty(fa.fa_fwd_host_device_bytes(B, H, N, d), dtype=torch.uint8, device="cuda")
    busy()
    fa.fa_fwd_host(*ins, torch.empty(SHAPE, dtype=torch.bfloat16).pin_memory(), torch.empty((B, H, N)).pin_memory(), False,
                   scale_f32(d), buf)
    held = scribble(6)
    torch.cuda.synchronize()
    assert all(t.isnan().all() for t in held)


def test_tensors_are_let_go_when_the_call_is_done():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, H, N, d = SHAPE
    x, _ = inputs(B, H, N, d, BASE_SEED + 1502)
    ins = [host_bf16(x[n], True) for n in ("q", "k", "v")]
    o, lse = torch.empty(SHAPE, dtype=torch.bfloat16).pin_memory(), torch.empty((B, H, N)).pin_memory()
    buf = torch.empty(fa.fa_fwd_host_device_bytes(B, H, N, d), dtype=torch.uint8, device="cuda")
    refs = [weakref.ref(t) for t in ins]
    busy()
    fa.fa_fwd_host(*ins, o, lse, False, scale_f32(d), buf)
    del ins
    assert all(r() is not None for r in refs)
    assert fa.fa_get_device_status() == 0
    assert all(r() is None for r in refs)
