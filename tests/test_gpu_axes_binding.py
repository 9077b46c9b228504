"""How the binding of the rotation by axes takes its axes and positions."""

import numpy as np
import pytest

import test_gpu_norm_rope as nr

pytestmark = pytest.mark.gpu

SEED, ROWS = 92000, 40


def case(seed):
    import torch
    x, _ = nr.packed(2, 9, 6, 64, seed)
    cos, sin, _, _ = nr.tables(ROWS, 64)
    pos = torch.tensor(np.random.default_rng(seed).integers(0, ROWS, (3, 2, 9)), dtype=torch.int32, device="cuda")
    return nr.split(x, 4, 1), cos, sin, pos


def test_axes_by_number():
    """An integer turned every pair by axis 0, and an array of 64-bit numbers was taken by its bytes."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    views, cos, sin, pos = case(SEED)
    axes = [i % 3 for i in range(32)]
    want = fa.norm_rope(*views, None, None, cos, sin, pos, axes=axes)
    for same in (bytes(axes), np.array(axes), np.array(axes, np.int32), torch.tensor(axes)):
        for x, y in zip(fa.norm_rope(*views, None, None, cos, sin, pos, axes=same), want):
            assert torch.equal(x, y)
    for bad in (32, np.int64(32), np.zeros(4, np.int64), np.zeros(8, np.int32)):
        with pytest.raises(ValueError):
            fa.norm_rope(*views, None, None, cos, sin, pos, axes=bad)
        with pytest.raises(ValueError):
            fa.norm_rope_backward(*want, *views[:2], None, None, cos, sin, pos, axes=bad)
    assert fa.fa_get_device_status() == 0


def test_the_calls_by_axes_need_axes():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    views, cos, sin, pos = case(SEED + 1)
    out = [torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in views]
    with pytest.raises(ValueError, match="axes"):
        fa.fa_norm_rope_axes_fwd(*views, None, None, cos, sin, pos[0].contiguous(), None, *out)
    with pytest.raises(ValueError, match="axes"):
        fa.fa_norm_rope_axes_bwd(*out, None, None, None, None, cos, sin, pos[0].contiguous(), None, *out, None, None, None)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in out)


@pytest.mark.parametrize("norm", [True, False])
def test_without_a_rotation_axes_and_positions_are_not_used(norm):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    views, _, _, pos = case(SEED + 2)
    w = nr.weights(64, SEED + 2, torch.float32)[0] if norm else None
    want = fa.norm_rope(*views, w, w)
    back = fa.norm_rope_backward(*want, *views[:2], w, w)
    for axes, p in (([], None), ([0] * 32, None), ([], pos)):
        for x, y in zip(fa.norm_rope(*views, w, w, None, None, p, axes=axes), want):
            assert torch.equal(x, y)
        got = fa.norm_rope_backward(*want, *views[:2], w, w, None, None, p, axes=axes)
        assert all(x is y is None or torch.equal(x, y) for x, y in zip(got, back))
    assert fa.fa_get_device_status() == 0
