"""CPU pins of the float64 oracle of the norm + rotation, the paged 8-bit cache
and the attention over it (oracle/cache_ops.py)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache_ops as co


def angles(pos, rot, base=10000.0):
    a = np.asarray(pos, dtype=np.float64)[..., None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32, 64])
def test_rotation_keeps_norms_and_depends_on_distance(rot, interleaved):
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 64))
    dots = []
    for p, q in ((3, 10), (103, 110)):
        a = co.rotate(x, *angles(p, rot), interleaved)
        b = co.rotate(y, *angles(q, rot), interleaved)
        assert abs(np.linalg.norm(a) - np.linalg.norm(x)) < 1e-12
        assert np.array_equal(a[rot:], x[rot:])
        dots.append(a @ b)
    assert abs(dots[0] - dots[1]) < 1e-12


def test_rotation_of_a_quarter_turn():
    x = np.arange(4.0)
    assert np.allclose(co.rotate(x, np.zeros(2), np.ones(2), True), [-1, 0, -3, 2])
    assert np.allclose(co.rotate(x, np.zeros(2), np.ones(2), False), [-2, -3, 0, 1])


def test_unit_weights_give_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((5, 64)) * 7
    y = co.norm_rope(x, np.ones(64), *angles(np.arange(5), 64), eps=0.0)
    assert np.allclose((y * y).mean(-1), 1, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_match_differences(norm, interleaved):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 4, 32))
    w = 1 + 0.3 * rng.standard_normal(32) if norm else None
    c, s = angles([0, 5, 9, 70], 16)
    dx, dw = co.norm_rope_backward(dy, x, w, c, s, interleaved, 1e-3)

    def loss(x_, w_):
        return float((co.norm_rope(x_, w_, c, s, interleaved, 1e-3) * dy).sum())

    for i, j in ((0, 0), (1, 7), (2, 15), (3, 31), (1, 16)):
        e = np.zeros_like(x)
        e[i, j] = 1e-5
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-5 - dx[i, j]) < 1e-8
    if norm:
        for j in (0, 9, 31):
            e = np.zeros(32)
            e[j] = 1e-5
            assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-5 - dw[j]) < 1e-8


def test_e4m3_codes_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(co.e4m3_values(), want.astype(np.float64), equal_nan=True)
    x = np.random.default_rng(4).standard_normal(20000).astype(np.float32) * np.float32(40)
    x = np.concatenate([x, x * np.float32(2 ** -12), np.float32([0, -0.0, 448, -448, 2 ** -10, 3 * 2 ** -10])])
    x = x[np.abs(x) <= 448]
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(co.to_e4m3(x), got)


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (0.0, 2.0 ** -100), (1.0, 2.0 ** -8),
                                       (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (3e38, 2.0 ** 120)])
def test_page_scale(amax, want):
    assert co.page_scale(amax) == want


def test_append_in_pieces_keeps_relative_error_and_reads_back():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((1, 2, 40, 64))
    code, scale = np.zeros((4, 2, 16, 64), np.uint8), np.zeros((4, 2))
    table = np.array([[2, 0, 3]])
    for lo, hi in ((0, 5), (5, 6), (6, 33), (33, 40)):
        code, scale = co.cache_append(x[:, :, lo:hi], code, scale, table, [hi], [hi - lo])
    got = co.cache_rows(code, scale, table[0], 40)
    # two roundings at most where a page's scale grew: half a step each, and the subnormal step 2^-9 of the scale
    tol = 2 * 2.0 ** -4 * np.abs(x[0]) + 2.0 ** -9 * scale.max()
    assert (np.abs(got - x[0]) <= tol).all()
    again, scale2 = co.cache_append(got[None][:, :, 32:40], code, scale, table, [40], [8])
    assert np.array_equal(again, code) and np.array_equal(scale2, scale)


@pytest.mark.parametrize("causal", [False, True])
def test_cache_attention_is_attention_over_the_rows(causal):
    rng = np.random.default_rng(6)
    B, Hq, Hkv, Nq, n, d = 2, 4, 2, 3, 21, 16
    q = rng.standard_normal((B, Hq, Nq, d))
    table = np.array([[1, 0], [3, 2]])
    pools = []
    for _ in range(2):
        x = rng.standard_normal((B, Hkv, n, d))
        pools += co.cache_append(x, np.zeros((4, Hkv, 16, d), np.uint8), np.zeros((4, Hkv)), table, [n] * B, [n] * B)
    o, lse = co.cache_attention(q, *pools, table, [n] * B, [Nq] * B, causal, 0.3)
    k = np.stack([co.cache_rows(pools[0], pools[1], table[b], n) for b in range(B)])
    v = np.stack([co.cache_rows(pools[2], pools[3], table[b], n) for b in range(B)])
    o_ref, l_ref = oracle.attention_forward(q, k, v, causal, 0.3)
    assert np.abs(o - o_ref).max() < 1e-12 and np.abs(lse - l_ref).max() < 1e-12


def test_cache_attention_rows_without_keys():
    q = np.ones((1, 1, 3, 16))
    z = np.zeros((1, 1, 16, 16), np.uint8), np.ones((1, 1))
    o, lse = co.cache_attention(q, *z, *z, np.zeros((1, 1), int), [1], [2], True, 1.0)
    assert lse[0, 0, 0] == -np.inf and (o[0, 0, 0] == 0).all() and lse[0, 0, 1] == 0 and np.isnan(lse[0, 0, 2])
