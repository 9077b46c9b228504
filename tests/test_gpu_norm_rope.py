"""GPU parity of the per-head norm with position rotation and its gradients
(fa_norm_rope_fwd / _bwd) against the float64 oracle on the same bf16 inputs.

Tolerances, per element: half a bf16 step of the exact value (2^-8 relative),
plus the fp32 work. A column of y is at most three products of rounded factors
(x r w, times cos or sin) and one sum; r carries the fp32 sum of d squares and
an rsqrt of 2 ulp. Together fewer than 32 roundings of 2^-24 relative to
|z_a| + |z_b|: 2^-19. A gradient adds the sum of d products h x (another
d / 8 + 5 additions in a lane and its group) against its own absolute terms:
2^-18 of r (|h| + |x| r^2 mean|h x|). dw adds at most a few hundred rows in a
lane and 32 groups in fp32: 2^-14 of the sum of absolute terms would already be
4 ulp a row; 2^-17 is taken for the rows here (at most 64 additions a chain).
"""

import numpy as np
import pytest

from attn_inputs import BASE_SEED, bf16_bits_to_f64, f32_to_bf16_bits
from gpu_util import to_device, to_host64
from oracle import cache_ops as co

pytestmark = pytest.mark.gpu

EPS = 1e-6


def packed(B, N, H, d, seed, spread=1.5):
    bits = f32_to_bf16_bits((np.random.default_rng(seed).standard_normal((B, N, H, d)) * spread).astype(np.float32))
    return to_device(bits), bf16_bits_to_f64(bits)


def tables(rows, rot):
    import exact_softmax_attention_fa_gb300 as fa
    if rot == 0:
        return None, None, np.ones((rows, 0)), np.zeros((rows, 0))
    c, s = fa.rope_tables(rows, rot)
    return c, s, c.double().cpu().numpy(), s.double().cpu().numpy()


def weights(d, seed, dtype):
    import torch
    if dtype is None:
        return None, None
    w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype)
    return w.cuda(), w.double().numpy()


def split(x, Hq, Hkv):
    """Views [B, H, N, d] of a packed [B, N, Hq + 2 Hkv, d] projection."""
    return x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2), x[:, :, Hq + Hkv:].transpose(1, 2)


def heads(x, Hq, Hkv):
    return [a.swapaxes(1, 2) for a in (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])]


def bound_fwd(x, w, cos, sin, inter, y):
    z = co.norm_rope(x, w, np.ones_like(cos), np.zeros_like(sin), inter, EPS)
    z, cos, sin = np.abs(z), np.abs(cos), np.abs(sin)
    mag = np.maximum(co.rotate(z, cos, sin, inter), co.rotate(z, cos, -sin, inter))  # |z_a c| + |z_b s|
    return 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * (mag + z) + 1e-37


CASES = [  # B, Hq, Hkv, N, d, rot, interleaved, weights
    (1, 1, 1, 1, 64, 64, False, "float32"),
    (2, 8, 2, 33, 128, 128, False, "float32"),
    (2, 8, 2, 33, 128, 128, True, "bfloat16"),
    (3, 6, 2, 17, 64, 32, True, "float32"),
    (1, 5, 1, 129, 64, 48, False, "bfloat16"),
    (2, 3, 3, 21, 256, 256, False, "float32"),
    (2, 16, 1, 7, 256, 16, True, None),
    (1, 4, 4, 40, 128, 96, False, None),
    (2, 9, 3, 5, 128, 0, False, "float32"),
    (1, 7, 0, 11, 128, 128, False, "float32"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("with_v", [True, False])
def test_forward(case, with_v):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d, rot, inter, wt = case
    wt = None if wt is None else getattr(torch, wt)
    x, f = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + N)
    cos, sin, c64, s64 = tables(500, rot)
    pos = np.random.default_rng(N).integers(0, 500, (B, N))
    (wq, wq64), (wk, wk64) = weights(d, 1, wt), weights(d, 2, wt)
    qi, ki, vi = split(x, Hq, Hkv)
    q, k, v = fa.norm_rope(qi, ki, vi if with_v else None, wq, wk, cos, sin,
                           torch.tensor(pos, dtype=torch.int32, device="cuda"), inter, EPS)
    assert fa.fa_get_device_status() == 0
    fq, fk, fv = heads(f, Hq, Hkv)
    c, s = c64[pos][:, None], s64[pos][:, None]
    for got, xin, w in ((q, fq, wq64), (k, fk, wk64)):
        y = co.norm_rope(xin, w, c, s, inter, EPS)
        err = np.abs(to_host64(got) - y)
        assert (err <= bound_fwd(xin, w, c, s, inter, y)).all(), err.max()
    if with_v:
        assert np.array_equal(to_host64(v), fv)
    else:
        assert v is None


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("with_v", [True, False])
def test_backward(case, with_v):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d, rot, inter, wt = case
    wt = None if wt is None else getattr(torch, wt)
    H = Hq + 2 * Hkv
    x, f = packed(B, N, H, d, BASE_SEED + 50 + N)
    dy, fdy = packed(B, N, H, d, BASE_SEED + 70 + N, 1.0)
    cos, sin, c64, s64 = tables(500, rot)
    pos = np.random.default_rng(N).integers(0, 500, (B, N))
    (wq, wq64), (wk, wk64) = weights(d, 3, wt), weights(d, 4, wt)
    qi, ki, _ = split(x, Hq, Hkv)
    dq, dk, dv = (t.contiguous() for t in split(dy, Hq, Hkv))
    grad = torch.full_like(x, 7.0)
    out = split(grad, Hq, Hkv)
    if not with_v:
        dv, out = None, (*out[:2], None)
    *_, dwq, dwk = fa.norm_rope_backward(dq, dk, dv, qi, ki, wq, wk, cos, sin,
                                         torch.tensor(pos, dtype=torch.int32, device="cuda"), out, inter, EPS)
    assert fa.fa_get_device_status() == 0
    c, s = c64[pos][:, None], s64[pos][:, None]
    got = heads(to_host64(grad), Hq, Hkv)
    xin, gin = heads(f, Hq, Hkv), heads(fdy, Hq, Hkv)
    for t, (w, dw) in enumerate(((wq64, dwq), (wk64, dwk))):
        dx_ref, dw_ref = co.norm_rope_backward(gin[t], xin[t], w, c, s, inter, EPS)
        ones = np.ones(d) if w is None else np.abs(w)
        g_abs = np.abs(co.rotate(np.abs(gin[t]), np.abs(c), -np.abs(s), inter)) + np.abs(gin[t])
        g_abs = np.maximum(g_abs, co.rotate(np.abs(gin[t]), np.abs(c), np.abs(s), inter))
        mag = g_abs
        if w is not None:
            r = 1 / np.sqrt((xin[t] ** 2).mean(-1, keepdims=True) + EPS)
            hx = (g_abs * ones * np.abs(xin[t])).mean(-1, keepdims=True)
            mag = r * (g_abs * ones + np.abs(xin[t]) * r * r * hx)
            terms = (g_abs * np.abs(xin[t]) * r).reshape(-1, d).sum(0)
            assert (np.abs(dw.double().cpu().numpy() - dw_ref) <= 2.0 ** -17 * terms + 1e-37).all()
        else:
            assert dw is None
        err = np.abs(got[t] - dx_ref)
        assert (err <= 2.0 ** -8 * np.abs(dx_ref) + 2.0 ** -18 * mag + 1e-37).all(), (t, err.max())
    assert np.array_equal(got[2], gin[2] if with_v else np.full_like(gin[2], 7.0))


def test_gradients_match_differences_of_the_forward():
    # the bf16 output rounds every difference, so the loss is taken along one
    # direction of w, whose gradient is a sum over all rows
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d = 2, 4, 2, 64, 64
    x, f = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 90)
    dy, fdy = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 91, 1.0)
    cos, sin, _, _ = tables(N, d)
    wq, wk = torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
    qi, ki, _ = split(x, Hq, Hkv)
    dq, dk, _ = (t.contiguous() for t in split(dy, Hq, Hkv))
    _, _, _, dwq, _ = fa.norm_rope_backward(dq, dk, None, qi, ki, wq, wk, cos, sin)
    step = torch.linspace(-1, 1, d, device="cuda")
    h = 0.25

    def loss(w):
        q, _, _ = fa.norm_rope(qi, ki, None, w, wk, cos, sin)
        return float((q.double() * dq.double()).sum())

    diff = (loss(1 + h * step) - loss(1 - h * step)) / (2 * h)  # the forward is linear in w
    # each output's rounding is independent: |y| 2^-9 rms at most, summed in squares with a factor 6
    tol = 6 * 2.0 ** -9 * float(dq.double().norm()) * 4 / (2 * h)
    assert abs(diff - float((dwq * step).sum())) <= tol


def test_contiguous_and_broadcast_inputs_and_default_positions():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    cos, sin, c64, s64 = tables(64, 128)
    x, f = packed(1, 64, 2, 128, BASE_SEED + 95)
    q = x.transpose(1, 2).contiguous()  # [1, 2, 64, 128]
    k = q[:, :1].expand(3, 4, 64, 128)  # batch and head strides of 0
    qq, kk, _ = fa.norm_rope(q.expand(3, 2, 64, 128), k, None, None, None, cos, sin)
    y = co.norm_rope(f.swapaxes(1, 2), None, c64[None, None], s64[None, None])
    tol = bound_fwd(f.swapaxes(1, 2), None, c64[None, None], s64[None, None], False, y)
    for b in range(3):
        assert (np.abs(to_host64(qq[b:b + 1]) - y) <= tol).all()
        for h in range(4):
            assert (np.abs(to_host64(kk[b, h]) - y[0, 0]) <= tol[0, 0]).all()


def test_far_positions_rotate_exactly():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    rows = 131072
    cos, sin = fa.rope_tables(rows, 64)
    a = (rows - 1) * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.abs(cos[-1].cpu().numpy() - np.cos(a)).max() <= 2.0 ** -24
    x, f = packed(1, 1, 3, 64, BASE_SEED + 96)
    qi, ki, vi = split(x, 1, 1)
    q, _, _ = fa.norm_rope(qi, ki, vi, None, None, cos, sin, torch.tensor([[rows - 1]], dtype=torch.int32, device="cuda"))
    y = co.norm_rope(f[:, :, 0], None, np.cos(a), np.sin(a))
    z = np.abs(f[:, :, 0])
    assert (np.abs(to_host64(q)[0] - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * (z + np.roll(z, 32, -1))).all()


def test_zero_rows_and_values_that_are_not_finite():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    x = torch.randn(1, 4, 3, 64, device="cuda").bfloat16()
    x[0, 0] = 0
    x[0, 1, 0, 5] = float("nan")
    x[0, 2, 0, 6] = float("inf")
    w = torch.ones(64, device="cuda")
    qi, ki, vi = split(x, 1, 1)
    q, k, v = fa.norm_rope(qi, ki, vi, w, w, *tables(4, 64)[:2])
    assert (q[0, 0, 0] == 0).all()
    assert q[0, 0, 1].isnan().all()  # the mean of a row with a NaN is NaN
    assert q[0, 0, 2].isnan().any() and torch.isfinite(q[0, 0, 3]).all()
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_positions_outside_the_tables_are_reported_and_leave_their_rows():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    x, f = packed(2, 5, 6, 64, BASE_SEED + 97)
    cos, sin, c64, s64 = tables(8, 64)
    pos = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    pos[0, 1], pos[1, 3], pos[1, 4] = -1, 8, 2 ** 31 - 1
    pos[1, :3] = 7
    qi, ki, vi = split(x, 4, 1)
    q, k, v = (torch.full((2, h, 5, 64), 3.0, device="cuda").bfloat16() for h in (4, 1, 1))
    fa.fa_norm_rope_fwd(qi, ki, vi, None, None, cos, sin, pos, q, k, v)
    code, where, _, _ = fa.fa_get_device_status_detail()
    assert (code, where) == (8, 21)
    bad = [(0, 1), (1, 3), (1, 4)]
    for b in range(2):
        for n in range(5):
            left = bool((q[b, :, n] == 3.0).all()) and bool((k[b, :, n] == 3.0).all())
            assert left == ((b, n) in bad)
    assert np.array_equal(to_host64(v), heads(f, 4, 1)[2])
    # backward: the same tokens add nothing to dw and leave their rows
    w = torch.ones(64, device="cuda")
    g = torch.full_like(x, 3.0)
    dq, dk = torch.randn(2, 4, 5, 64, device="cuda").bfloat16(), torch.randn(2, 1, 5, 64, device="cuda").bfloat16()
    *_, dwq, _ = fa.norm_rope_backward(dq, dk, None, qi, ki, w, w, cos, sin, pos, (*split(g, 4, 1)[:2], None))
    assert fa.fa_get_device_status_detail()[:2] == (8, 22)
    assert fa.fa_get_device_status() == 0
    for b, n in bad:
        assert (g[b, n] == 3.0).all()
        dq[b, :, n] = 0
    good = pos.clamp(0, 7)
    *_, dw2, _ = fa.norm_rope_backward(dq, dk, None, qi, ki, w, w, cos, sin, good)
    assert torch.equal(dwq, dw2)


def test_backward_is_bitwise_reproducible_and_replays_from_a_graph():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d = 2, 8, 2, 700, 128
    x, _ = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 98)
    cos, sin, _, _ = tables(N, d)
    w = torch.ones(d, device="cuda")
    qi, ki, vi = split(x, Hq, Hkv)
    q, k, v = (torch.empty(B, h, N, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    grad = torch.empty_like(x)
    dwq, dwk = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(B, Hq, Hkv, N, d), dtype=torch.uint8, device="cuda")

    def step():
        fa.fa_norm_rope_fwd(qi, ki, vi, w, w, cos, sin, None, q, k, v)
        fa.fa_norm_rope_bwd(q, k, v, qi, ki, w, w, cos, sin, None, *split(grad, Hq, Hkv), dwq, dwk, ws)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (q, k, v, grad, dwq, dwk)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for t in (q, k, v, grad, dwq, dwk):
            t.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (q, k, v, grad, dwq, dwk)))


def test_training_step_through_the_attention():
    """projection -> norm + rotation -> attention -> loss, and back to the
    packed projection's gradient, against the oracle's chain on the same bf16
    tensors (each kernel's bf16 outputs are the next one's inputs)."""
    import exact_softmax_attention_fa_gb300 as fa
    import oracle
    import torch
    from gpu_util import TOL_GRAD_REL, TOL_O, scale_f32
    B, Hq, Hkv, N, d = 1, 4, 2, 150, 64
    x, f = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 99)
    cos, sin, c64, s64 = tables(N, d)
    (wq, wq64), (wk, wk64) = weights(d, 5, torch.float32), weights(d, 6, torch.float32)
    qi, ki, vi = split(x, Hq, Hkv)
    q, k, v = fa.norm_rope(qi, ki, vi, wq, wk, cos, sin)
    o, lse = fa.forward(q, k, v, causal=True)
    do = torch.randn(o.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    dq, dk, dv = fa.backward(q, k, v, o, lse, do, causal=True)
    grad = torch.empty_like(x)
    *_, dwq, dwk = fa.norm_rope_backward(dq, dk, dv, qi, ki, wq, wk, cos, sin, None, split(grad, Hq, Hkv))
    assert fa.fa_get_device_status() == 0
    scale = scale_f32(d)
    xin = heads(f, Hq, Hkv)
    q64 = co.norm_rope(xin[0], wq64, c64, s64, eps=EPS)
    k64 = co.norm_rope(xin[1], wk64, c64, s64, eps=EPS)
    o64, _ = oracle.attention_forward(q64, k64, xin[2], True, scale)
    g64 = oracle.attention_backward(q64, k64, xin[2], to_host64(do), True, scale)
    # q and k reach the attention rounded to bf16: the parity bars of the
    # attention, once more for that rounding
    assert np.abs(to_host64(o) - o64).max() <= 2 * TOL_O
    got = heads(to_host64(grad), Hq, Hkv)
    for t, w in ((0, wq64), (1, wk64)):
        ref, dw_ref = co.norm_rope_backward(g64[t], xin[t], w, c64, s64, eps=EPS)
        assert np.abs(got[t] - ref).max() <= 2 * TOL_GRAD_REL * np.abs(ref).max()
        dw = (dwq, dwk)[t].double().cpu().numpy()
        assert np.abs(dw - dw_ref).max() <= 2 * TOL_GRAD_REL * np.abs(dw_ref).max()
    assert np.abs(got[2] - g64[2]).max() <= TOL_GRAD_REL * np.abs(g64[2]).max()
