"""GPU parity of the norm and rotation on batches in which a lane group of the backward
takes several units: the persistent loop's stride, the angles it loads again and the
weight gradients it sums over units, against the float64 oracle.

Tolerances as in test_gpu_norm_rope.py. A weight gradient's lane adds at most 8 rows of
each of its units (16 units at most here: 128 additions) and the block 32 groups, each
term of at most 8 roundings: 168 * 2^-24 < 2^-16 of the sum of absolute terms.
"""

import numpy as np
import pytest

from attn_inputs import BASE_SEED
from gpu_util import to_host64
from oracle import cache_ops as co
from test_gpu_norm_rope import EPS, bound_fwd, heads, packed, split, tables, weights

pytestmark = pytest.mark.gpu

CASES = [  # B, Hq, Hkv, N, d, rot, interleaved, weights
    (2, 9, 3, 3001, 128, 128, False, "float32"),
    (2, 9, 3, 3001, 128, 96, True, "bfloat16"),
    (2, 9, 3, 1501, 256, 256, False, "float32"),
    (1, 4, 1, 20011, 64, 32, True, "float32"),
    (2, 9, 3, 3001, 128, 128, False, None),
    (3, 12, 0, 2003, 256, 64, False, "bfloat16"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("with_v", [True, False])
def test_both_directions(case, with_v):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, N, d, rot, inter, wt = case
    groups = 256 // (d // 8)  # lane groups of a block; at most 304 blocks in all
    assert B * N * -(-Hq // 8) > 304 * groups  # each takes more than one unit of 8 heads of a token
    assert B * N * -(-Hq // 8) / (304 * groups * Hq / (Hq + 2 * Hkv) * 0.75) < 16
    wt = None if wt is None else getattr(torch, wt)
    x, f = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + N)
    dy, fdy = packed(B, N, Hq + 2 * Hkv, d, BASE_SEED + N + 1, 1.0)
    cos, sin, c64, s64 = tables(5000, rot)
    pos = np.random.default_rng(N).integers(0, 5000, (B, N))
    dev_pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    (wq, wq64), (wk, wk64) = weights(d, 1, wt), weights(d, 2, wt)
    qi, ki, vi = split(x, Hq, Hkv)
    xin, gin = heads(f, Hq, Hkv), heads(fdy, Hq, Hkv)
    c, s = c64[pos][:, None], s64[pos][:, None]

    q, k, v = fa.norm_rope(qi, ki, vi if with_v else None, wq, wk, cos, sin, dev_pos, inter, EPS)
    assert fa.fa_get_device_status() == 0
    for got, t, w in ((q, 0, wq64), (k, 1, wk64)):
        y = co.norm_rope(xin[t], w, c, s, inter, EPS)
        assert (np.abs(to_host64(got) - y) <= bound_fwd(xin[t], w, c, s, inter, y)).all()
    assert v is None if not with_v else np.array_equal(to_host64(v), xin[2])

    dq, dk, dv = (t.contiguous() for t in split(dy, Hq, Hkv))
    grad = torch.full_like(x, 7.0)
    out = split(grad, Hq, Hkv)
    if not with_v:
        dv, out = None, (*out[:2], None)
    *_, dwq, dwk = fa.norm_rope_backward(dq, dk, dv, qi, ki, wq, wk, cos, sin, dev_pos, out, inter, EPS)
    assert fa.fa_get_device_status() == 0
    got = heads(to_host64(grad), Hq, Hkv)
    for t, (w, dw) in enumerate(((wq64, dwq), (wk64, dwk))):
        dx_ref, dw_ref = co.norm_rope_backward(gin[t], xin[t], w, c, s, inter, EPS)
        g = np.abs(gin[t])
        mag = np.maximum(co.rotate(g, np.abs(c), np.abs(s), inter), np.abs(co.rotate(g, np.abs(c), -np.abs(s), inter)) + g)
        if w is not None:
            r = 1 / np.sqrt((xin[t] ** 2).mean(-1, keepdims=True) + EPS)
            terms = (mag * np.abs(xin[t]) * r).reshape(-1, d).sum(0)
            assert (np.abs(dw.double().cpu().numpy() - dw_ref) <= 2.0 ** -16 * terms + 1e-37).all(), t
            hx = (mag * np.abs(w) * np.abs(xin[t])).mean(-1, keepdims=True)
            mag = r * (mag * np.abs(w) + np.abs(xin[t]) * r * r * hx)
        else:
            assert dw is None
        err = np.abs(got[t] - dx_ref)
        assert (err <= 2.0 ** -8 * np.abs(dx_ref) + 2.0 ** -18 * mag + 1e-37).all(), (t, err.max())
    assert np.array_equal(got[2], gin[2] if with_v else np.full_like(gin[2], 7.0))
