"""GPU parity of the norm with the rotation by several axes (fa_norm_rope_axes_fwd / _bwd) against the float64 oracle,
with the angles of every token's pairs gathered on the host; the bounds are those of test_gpu_norm_rope. And the
whole run on packed sequences: projection, norm and rotation, attention, and back into the projection's gradient."""

import numpy as np
import pytest

import test_gpu_norm_rope as nr
from attn_inputs import BASE_SEED
from gpu_util import scale_f32, to_host64
from oracle import cache_ops as co

pytestmark = pytest.mark.gpu

FA_ERR_INDEX = 8
ROWS = 500


def blocks(*n):
    return [a for a, m in enumerate(n) for _ in range(m)]


CASES = [  # B, Hq, Hkv, N, d, the axis of each pair, interleaved, weights
    (1, 1, 1, 1, 64, blocks(32), False, "float32"),
    (2, 8, 2, 33, 128, blocks(16, 24, 24), False, "float32"),
    (2, 8, 2, 33, 128, blocks(16, 24, 24), True, "bfloat16"),
    (2, 5, 1, 41, 128, [i % 3 for i in range(64)], False, "float32"),
    (1, 5, 1, 129, 64, [i % 2 for i in range(24)], True, "float32"),
    (3, 4, 2, 17, 64, blocks(5, 6, 2, 3), False, None),
    (2, 3, 3, 21, 256, [(7 * i) % 4 for i in range(128)], False, "bfloat16"),
    (1, 9, 3, 70, 256, blocks(1, 127), True, "float32"),
    (2, 7, 0, 11, 128, blocks(3, 29, 32), False, "float32"),
    (16, 32, 8, 1, 128, blocks(16, 24, 24), False, "float32"),
    # tokens of several units with different numbers of heads beside each other in a warp
    (2, 20, 3, 97, 64, [i % 3 for i in range(32)], False, "float32"),
    (1, 13, 11, 600, 64, blocks(10, 22), True, "bfloat16"),
    (3, 20, 9, 203, 128, blocks(64), False, "float32"),
    # five units and more for each of the lane groups of 304 blocks: the backward's ring
    (1, 1, 1, 4100, 256, blocks(1, 127), True, "float32"),
    (2, 1, 1, 4100, 128, [i % 3 for i in range(64)], False, "bfloat16"),
    (1, 20, 3, 9800, 64, [i % 2 for i in range(24)], False, "float32"),
    (1, 1, 1, 8200, 128, blocks(20, 44), False, None),
]


def setup(case, seed):
    import torch
    B, Hq, Hkv, N, d, axes, inter, wt = case
    pos = np.random.default_rng(seed).integers(0, ROWS, (max(axes) + 1, B, N))
    cos, sin, c64, s64 = nr.tables(ROWS, 2 * len(axes))
    at = [c64[pos[a], i] for i, a in enumerate(axes)], [s64[pos[a], i] for i, a in enumerate(axes)]
    c, s = (np.stack(x, -1)[:, None] for x in at)  # [B, 1, N, rot / 2]
    return pos, torch.tensor(pos, dtype=torch.int32, device="cuda"), cos, sin, c, s


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d, axes, inter, wt = case
    wt = None if wt is None else getattr(torch, wt)
    x, f = nr.packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 300 + N)
    _, pos, cos, sin, c, s = setup(case, N)
    (wq, wq64), (wk, wk64) = nr.weights(d, 1, wt), nr.weights(d, 2, wt)
    q, k, v = fa.norm_rope(*nr.split(x, Hq, Hkv), wq, wk, cos, sin, pos, inter, nr.EPS, axes=axes)
    assert fa.fa_get_device_status() == 0
    fq, fk, fv = nr.heads(f, Hq, Hkv)
    for got, xin, w in ((q, fq, wq64), (k, fk, wk64)):
        y = co.norm_rope(xin, w, c, s, inter, nr.EPS)
        assert (np.abs(to_host64(got) - y) <= nr.bound_fwd(xin, w, c, s, inter, y)).all()
    assert np.array_equal(to_host64(v), fv)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d, axes, inter, wt = case
    wt = None if wt is None else getattr(torch, wt)
    x, f = nr.packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 350 + N)
    dy, fdy = nr.packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + 370 + N, 1.0)
    _, pos, cos, sin, c, s = setup(case, N)
    (wq, wq64), (wk, wk64) = nr.weights(d, 3, wt), nr.weights(d, 4, wt)
    qi, ki, _ = nr.split(x, Hq, Hkv)
    grad = torch.full_like(x, 7.0)
    *_, dwq, dwk = fa.norm_rope_backward(*(t.contiguous() for t in nr.split(dy, Hq, Hkv)), qi, ki, wq, wk, cos, sin, pos,
                                         nr.split(grad, Hq, Hkv), inter, nr.EPS, axes=bytes(axes))
    assert fa.fa_get_device_status() == 0
    got, xin, gin = nr.heads(to_host64(grad), Hq, Hkv), nr.heads(f, Hq, Hkv), nr.heads(fdy, Hq, Hkv)
    for t, (w, dw) in enumerate(((wq64, dwq), (wk64, dwk))):
        dx_ref, dw_ref = co.norm_rope_backward(gin[t], xin[t], w, c, s, inter, nr.EPS)
        g_abs = np.maximum(co.rotate(np.abs(gin[t]), np.abs(c), -np.abs(s), inter),
                           co.rotate(np.abs(gin[t]), np.abs(c), np.abs(s), inter))
        g_abs = np.abs(g_abs) + np.abs(gin[t])
        mag = g_abs
        if w is not None:
            r = 1 / np.sqrt((xin[t] ** 2).mean(-1, keepdims=True) + nr.EPS)
            hx = (g_abs * np.abs(w) * np.abs(xin[t])).mean(-1, keepdims=True)
            mag = r * (g_abs * np.abs(w) + np.abs(xin[t]) * r * r * hx)
            terms = (g_abs * np.abs(xin[t]) * r).reshape(-1, d).sum(0)
            assert (np.abs(dw.double().cpu().numpy() - dw_ref) <= 2.0 ** -17 * terms + 1e-37).all()
        assert (np.abs(got[t] - dx_ref) <= 2.0 ** -8 * np.abs(dx_ref) + 2.0 ** -18 * mag + 1e-37).all(), t
    assert np.array_equal(got[2], gin[2])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_equal_positions_are_the_rotation_by_one(d, inter):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    x, _ = nr.packed(2, 19, 6, d, BASE_SEED + 400)
    cos, sin, _, _ = nr.tables(ROWS, d)
    w, _ = nr.weights(d, 1, torch.float32)
    pos = torch.randint(0, ROWS, (2, 19), dtype=torch.int32, device="cuda")
    axes = [(i // 3) % 3 for i in range(d // 2)]
    one = fa.norm_rope(*nr.split(x, 4, 1), w, w, cos, sin, pos, inter)
    by_axes = fa.norm_rope(*nr.split(x, 4, 1), w, w, cos, sin, pos.expand(3, 2, 19).contiguous(), inter, axes=axes)
    for a, b in zip(one, by_axes):
        assert torch.equal(a, b)
    args = [t.contiguous() for t in nr.split(x, 4, 1)], nr.split(x, 4, 1)[:2]
    one = fa.norm_rope_backward(*args[0], *args[1], w, w, cos, sin, pos, None, inter)
    by_axes = fa.norm_rope_backward(*args[0], *args[1], w, w, cos, sin, pos.expand(3, 2, 19).contiguous(), None, inter,
                                    axes=axes)
    for a, b in zip(one, by_axes):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [-1, ROWS, 2**31 - 1, -2**31])
@pytest.mark.parametrize("axis", [0, 1, 2])
def test_a_position_outside_the_tables_on_any_axis(axis, bad):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    x, _ = nr.packed(2, 9, 6, 64, BASE_SEED + 410)
    cos, sin, _, _ = nr.tables(ROWS, 64)
    pos = torch.randint(0, ROWS, (3, 2, 9), dtype=torch.int32, device="cuda")
    axes = blocks(10, 12, 10)
    good = fa.norm_rope(*nr.split(x, 4, 1), None, None, cos, sin, pos, axes=axes)
    assert fa.fa_get_device_status() == 0
    pos[axis, 1, 4] = bad
    q, k, v = (torch.full_like(t, 7.0) for t in good)
    fa.fa_norm_rope_axes_fwd(*nr.split(x, 4, 1), None, None, cos, sin, pos, axes, q, k, v)
    assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 21)
    hit = torch.zeros(2, 1, 9, 1, dtype=torch.bool, device="cuda")
    hit[1, 0, 4] = True
    for got, want in ((q, good[0]), (k, good[1])):
        assert torch.equal(got, torch.where(hit, torch.full_like(want, 7.0), want))
    assert torch.equal(v, good[2])
    out = [torch.full_like(t, 7.0) for t in good]
    fa.fa_norm_rope_axes_bwd(q, k, v, None, None, None, None, cos, sin, pos, axes, *out, None, None, None)
    assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 22)
    assert (out[0][1, :, 4] == 7).all() and (out[1][1, :, 4] == 7).all()


@pytest.mark.parametrize("norm", [True, False])
def test_a_position_outside_the_tables_among_many(norm):
    """As above in the backward for many units: the other tokens' gradients stay, the weights' sums leave it out."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    N, d, axes = 4100, 256, bytes([i % 2 for i in range(128)])
    x, _ = nr.packed(1, N, 3, d, BASE_SEED + 420)
    dy, _ = nr.packed(1, N, 3, d, BASE_SEED + 421, 1.0)
    cos, sin, _, _ = nr.tables(ROWS, d)
    pos = torch.randint(0, ROWS, (2, 1, N), dtype=torch.int32, device="cuda")
    (wq, _), (wk, _) = nr.weights(d, 3, torch.float32), nr.weights(d, 4, torch.float32)
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[[0, 1, 700, 2431, 2432, 4099]] = True

    def run(dy, pos):
        g = [t.contiguous() for t in nr.split(dy, 1, 1)]
        out = [torch.full_like(t, 7.0) for t in g]
        q, k, _ = nr.split(x, 1, 1)
        *_, dwq, dwk = fa.norm_rope_backward(*g, q if norm else None, k if norm else None, wq if norm else None,
                                             wk if norm else None, cos, sin, pos, out, axes=axes)
        return out, dwq, dwk

    zeroed = dy.clone()
    nr.split(zeroed, 1, 1)[0][0, 0, bad] = 0  # tokens whose gradient is nothing add nothing
    nr.split(zeroed, 1, 1)[1][0, 0, bad] = 0
    want, dwq, dwk = run(zeroed, pos)
    assert fa.fa_get_device_status() == 0
    pos[1, 0, bad] = ROWS
    got, bad_q, bad_k = run(dy, pos)
    assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 22)
    for t in range(2):
        assert (got[t][0, 0, bad] == 7).all() and torch.equal(got[t][0, 0, ~bad], want[t][0, 0, ~bad])
    assert torch.equal(got[2], nr.split(dy, 1, 1)[2])
    if norm:
        assert torch.equal(bad_q, dwq) and torch.equal(bad_k, dwk)


def test_binding_refuses():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    x, _ = nr.packed(2, 9, 6, 64, BASE_SEED + 420)
    cos, sin, _, _ = nr.tables(ROWS, 64)
    pos = torch.zeros(3, 2, 9, dtype=torch.int32, device="cuda")
    axes = blocks(10, 12, 10)
    call = lambda pos=pos, axes=axes: fa.norm_rope(*nr.split(x, 4, 1), None, None, cos, sin, pos, axes=axes)
    call()
    for bad in (dict(pos=None), dict(pos=pos[0]), dict(pos=pos.long()), dict(pos=pos[:, :1]), dict(pos=pos.transpose(1, 2)),
                dict(axes=axes[:-1]), dict(axes=axes + [0]), dict(axes=[-1] * 32), dict(axes=[256] * 32)):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(axes=[3] * 32), dict(pos=pos[:1]), dict(pos=pos[:0]),
                dict(pos=torch.zeros(5, 2, 9, dtype=torch.int32, device="cuda"))):
        with pytest.raises(fa.FAError):
            call(**bad)
    with pytest.raises(ValueError):  # positions of one axis alone, without axes
        fa.norm_rope(*nr.split(x, 4, 1), None, None, cos, sin, pos)
    assert fa.fa_get_device_status() == 0


def test_packed_step_from_projection_to_its_gradient():
    """Norm and rotation by time, height and width, packed attention and back, against the same chain in 64 bits.

    Bars: every stage is held to its own bound elsewhere; here the chain's outputs are held to 2% of their
    largest entry (the parity bar of the gradients), which a mixed up head, sequence or axis exceeds at once."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    lens, Hq, Hkv, d, axes = [70, 1, 131, 200], 4, 2, 64, blocks(8, 12, 12)
    T, H = sum(lens), Hq + 2 * Hkv
    x, f = nr.packed(1, T, H, d, BASE_SEED + 430)
    do, fdo = nr.packed(1, T, Hq, d, BASE_SEED + 431, 1.0)
    pos = np.random.default_rng(1).integers(0, ROWS, (3, 1, T))
    d_pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    cos, sin, c64, s64 = nr.tables(ROWS, d)
    w, w64 = nr.weights(d, 1, torch.float32)
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    plan, scale = fa.PackedPlan(cu, T), scale_f32(d)
    views = nr.split(x, Hq, Hkv)
    q, k, v = fa.norm_rope(*views, w, w, cos, sin, d_pos, axes=axes)
    qp, kp, vp = (t[0].transpose(0, 1) for t in (q, k, v))  # [T, H, d] views: nothing is copied
    o, lse = fa.forward_packed(qp, kp, vp, plan, scale=scale)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    fa.backward_packed(qp, kp, vp, o, lse, do[0], plan, scale=scale, out=[t[0].transpose(0, 1) for t in grads])
    dx = torch.empty_like(x)
    *_, dwq, dwk = fa.norm_rope_backward(*grads, *views[:2], w, w, cos, sin, d_pos, nr.split(dx, Hq, Hkv), axes=axes)
    assert fa.fa_get_device_status() == 0

    # the chain in 64 bits, by automatic differentiation
    t = torch.tensor(f, requires_grad=True)
    wt = torch.tensor(w64, requires_grad=True)
    c, s = (torch.tensor(np.stack([tab[pos[a], i] for i, a in enumerate(axes)], -1))[:, None] for tab in (c64, s64))

    def turn(z, w):
        z = z.transpose(1, 2)
        z = z / (z.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = z[..., :d // 2], z[..., d // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)[0]

    qr, kr = turn(t[:, :, :Hq], wt), turn(t[:, :, Hq:Hq + Hkv], wt)
    vr = t[0, :, Hq + Hkv:].transpose(0, 1)
    out = []
    for a, b in zip(np.cumsum([0] + lens), np.cumsum(lens)):
        kk, vv = (z[:, a:b].repeat_interleave(Hq // Hkv, 0) for z in (kr, vr))
        sc = qr[:, a:b] @ kk.transpose(1, 2) * scale
        sc = sc.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), float("-inf"))
        out.append(torch.softmax(sc, -1) @ vv)
    ref = torch.cat(out, 1).transpose(0, 1)
    (ref * torch.tensor(fdo[0])).sum().backward()
    for name, got, want in (("o", o, ref), ("dx", dx[0], t.grad[0]), ("dw", dwq + dwk, wt.grad)):
        want = want.detach().numpy()
        err = np.abs(got.double().cpu().numpy().reshape(want.shape) - want).max() / np.abs(want).max()
        assert err <= 2e-2, (name, err)
