"""GPU parity of fa_fwd_kv8 for every value scale a cache may hold: up to 2^126, down
to the smallest normal number, below it and 0, not powers of two, and pages whose
scales differ by more than fp32's range, in every order, in a warp's or CTA's run and
between runs. Against float64 on the same codes and scales.

Tolerances as in test_gpu_fwd_kv8.py: with p the exact weights, s the value scales,
e the pieces' error of a query value over its row's largest (2^-21 up to 16 rows per
K/V head, 2^-17 above), n keys and
  delta = scale max_j ((d/16 + 4) 2^-22 sum |q k_j| + e max|q| sum |k_j|) + 2^-22 E,
E the largest |t_j log2(e)| + |log2 s_j| (the exponent they share is rounded to fp32,
and the sum's exponent is taken from it):
  |O - O_ref| <= 2^-8 |O_ref| + A (2^-11 + 2^-20 + n 2^-24 + 2 delta)
                 + 2^-24 max_j(p_j s_j) sum_j |code_j| + 2^-133
                 + 448 (2^-100 + 2^-89 max_j s_j)
  |L - L_ref| <= delta + 2^-20 + 2 n 2^-24 + 2^-21 |L_ref|.
(2^-133: half a step of a subnormal bf16. The last term: a scale below 2^-100, or below
2^-90 of a larger one's power of two, counts as that; a power of two may be half
the scale. 2 n: weights below 2^-24 of the largest may leave fp32's range.)
"""

import numpy as np
import pytest

from attn_inputs import BASE_SEED, bf16_bits_to_f64, f32_to_bf16_bits
from gpu_util import scale_f32, to_device, to_host64
from kv8_util import ints
from oracle import cache_ops as co

pytestmark = pytest.mark.gpu


def run(q_bits, q, code, k_scale, v_scale, page, n, scale, causal=False):
    """One sequence of n keys, one K/V head, pages in order; every row against float64."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    _, Hq, Nq, d = q.shape
    pages = len(k_scale)
    dev = [torch.from_numpy(c.reshape(pages, 1, page, d)).cuda() for c in code]
    sc = [torch.from_numpy(np.asarray(s, dtype=np.float32).reshape(pages, 1)).cuda() for s in (k_scale, v_scale)]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    o = torch.full((1, Hq, Nq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, Hq, Nq), 5.0, device="cuda")
    ws = torch.full((fa.fa_fwd_kv8_workspace_size(1, Hq, 1, Nq, d),), 255, dtype=torch.uint8, device="cuda")
    fa.fa_fwd_kv8(to_device(q_bits), *dev, *sc, table, ints(n), o, lse, causal, scale, None, ws)
    assert fa.fa_get_device_status() == 0
    o, lse = to_host64(o)[0], lse.double().cpu().numpy()[0]
    sk, sv = (np.repeat(np.asarray(s, np.float32).astype(np.float64), page)[:n, None] for s in (k_scale, v_scale))
    k, v8 = (co.from_e4m3(c.reshape(-1, d)[:n]) for c in code)
    k, v = k * sk, v8 * sv
    see = np.arange(n)[None, :] < ((n - Nq + 1 + np.arange(Nq))[:, None] if causal else n)
    e_q = 2.0 ** -21 if Hq * Nq <= (8 if d == 256 else 16) else 2.0 ** -17
    for h in range(Hq):
        t = np.where(see, scale * (q[0, h] @ k.T), -np.inf)
        top = t.max(1, keepdims=True)
        e = np.exp(t - top)
        l = e.sum(1, keepdims=True)
        p, l_ref = e / l, (top + np.log(l))[:, 0]
        aq = np.abs(q[0, h])
        mag = scale * ((d / 16 + 4) * 2.0 ** -22 * (aq @ np.abs(k).T) +
                       e_q * aq.max(1)[:, None] * np.abs(k).sum(1)[None, :])
        E = np.abs(np.where(see, t, 0)).max(1) * 1.4427 + np.abs(np.log2(np.maximum(sv, 2.0 ** -100))).max()
        delta = np.where(see, mag, 0).max(1) + 2.0 ** -22 * E
        err_l = np.abs(lse[h] - l_ref)
        assert (err_l <= delta + 2.0 ** -20 + 2 * n * 2.0 ** -24 + 2.0 ** -21 * np.abs(l_ref)).all(), (h, err_l.max())
        o_ref, A = p @ v, p @ np.abs(v)
        tol = 2.0 ** -8 * np.abs(o_ref) + A * (2.0 ** -11 + 2.0 ** -20 + n * 2.0 ** -24 + 2 * delta[:, None]) + 2.0 ** -133
        tol += 2.0 ** -24 * (p * sv[:, 0]).max(1)[:, None] * (see @ np.abs(v8))
        tol += 448 * (2.0 ** -100 + 2.0 ** -89 * sv.max())
        err = np.abs(o[h] - o_ref)
        assert (err <= tol).all(), (h, err.max(), (err - tol).max(), np.abs(o_ref).max())


def tokens(rng, pages, page, d):
    """Codes of both pools, values of either sign from 2^-6 to 15."""
    return [co.to_e4m3(rng.standard_normal((pages * page, d)) * 3).astype(np.uint8) for _ in range(2)]


def queries(rng, Hq, Nq, d, spread=1.0):
    bits = f32_to_bf16_bits((rng.standard_normal((1, Hq, Nq, d)) * spread).astype(np.float32))
    return bits, bf16_bits_to_f64(bits)


ROWS = [(4, 1), (8, 2), (4, 20), (3, 100)]  # 4 and 16 rows; one tile, two tiles of rows


@pytest.mark.parametrize("Hq,Nq", ROWS)
@pytest.mark.parametrize("d,exp", [(d, e) for d in (64, 128) for e in (-np.inf, -140, -126, -120, -101, -100, 121, 126)] +
                         [(256, e) for e in (-np.inf, -126, 126)])
def test_many_equal_weights_at_the_ends_of_the_scales_range(d, exp, Hq, Nq):
    # 4096 keys of the same score: their sum is 2^12 whatever the scale is
    rng = np.random.default_rng(BASE_SEED + int(max(exp, -200)) + 200)
    pages, page = 64, 64
    code = tokens(rng, pages, page, d)
    if exp > 100:
        code[1] = (code[1] & 0x80) | (code[1] & 0x07)  # so that O stays in bf16's range
    bits, q = queries(rng, Hq, Nq, d, 0.0)
    run(bits, q, code, np.full(pages, 2.0 ** -4), np.full(pages, 2.0 ** exp), page, 4096, scale_f32(d))


ORDERS = {
    "rising": lambda i, n: i / (n - 1),
    "falling": lambda i, n: 1 - i / (n - 1),
    "mixed": lambda i, n: (i * 7 % n) / (n - 1),
    "two": lambda i, n: float(i % 2),
    "late": lambda i, n: float(i > n // 2),
    "early": lambda i, n: float(i <= n // 2),
}


@pytest.mark.parametrize("Hq,Nq", ROWS)
@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("n,lo,hi", [(330, -126, 110), (330, -100, -8), (330, -100, 0), (330, -100, 60), (330, 0, 120),
                                     (20000, -100, 60)])  # the last: parts that several SMs join
def test_pages_whose_value_scales_lie_far_apart(n, lo, hi, order, Hq, Nq):
    d, page = (64, 16) if n < 1000 else (128, 64)
    rng = np.random.default_rng(BASE_SEED + n + lo + hi + Hq)
    pages = -(-n // page)
    code = tokens(rng, pages, page, d)
    if hi > 100:
        code[1] = (code[1] & 0x80) | (code[1] & 0x07)
    bits, q = queries(rng, Hq, Nq, d)
    sv = np.exp2([round(lo + (hi - lo) * ORDERS[order](i, pages)) for i in range(pages)])
    run(bits, q, code, np.exp2(rng.integers(-5, -2, pages)), sv, page, n, scale_f32(d), causal=True)


@pytest.mark.parametrize("Hq,Nq", ROWS)
@pytest.mark.parametrize("spread", [0, 40, 110])
def test_scales_that_are_not_powers_of_two(spread, Hq, Nq):
    d, page, n = 128, 32, 3000
    rng = np.random.default_rng(BASE_SEED + spread)
    pages = -(-n // page)
    code = tokens(rng, pages, page, d)
    bits, q = queries(rng, Hq, Nq, d)
    sk, sv = (rng.uniform(1, 2, pages) for _ in range(2))
    run(bits, q, code, sk * 2.0 ** -4, sv * np.exp2(rng.integers(-spread, 1, pages)), page, n, scale_f32(d), causal=True)


@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_zero_values_beside_large_ones_written_by_the_cache(d, Nq):
    """The cache gives a page of zeros its smallest scale, 2^-100; half of the weight lies there."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    n = 1024
    for size in (1.0, 2.0 ** 30, 2.0 ** 90):
        for zero in (slice(0, n // 2), slice(n // 2, n)):
            cache = fa.KV8Cache(1, 1, d, n, page=64)
            k = torch.zeros(1, 1, n, d, dtype=torch.bfloat16, device="cuda")
            v = torch.full_like(k, size)
            v[:, :, zero] = 0
            cache.append(k, v)
            q = torch.randn(1, 4, Nq, d, device="cuda").bfloat16()
            o, lse = cache.attend(q, causal=False)
            assert fa.fa_get_device_status() == 0
            # equal weights: half of the keys hold `size` (exact in e4m3), and 2^-11 covers fp16 weights and their sum
            assert float((o.double() / size - 0.5).abs().max()) <= 2.0 ** -9
            assert float((lse.double() - np.log(n)).abs().max()) <= 2.0 ** -18 * np.log(n)


@pytest.mark.parametrize("Hq,Nq", [(1, 1), (4, 20)])
def test_a_sequence_of_small_values_behind_one_of_large_ones(Hq, Nq):
    """The largest scale of one sequence or head is of no effect on the next one in the same run."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hkv, d, n = 4, 2, 64, 200
    cache = fa.KV8Cache(B, Hkv, d, n, page=16)
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED)
    k, v = (torch.randn(B, Hkv, n, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    size = torch.tensor([[2.0 ** 100, 2.0 ** -60], [2.0 ** -80, 2.0 ** 70], [2.0 ** -70, 2.0 ** -85], [1.0, 2.0 ** -84]],
                        device="cuda")[..., None, None]
    q = torch.randn(B, Hkv * Hq, Nq, d, generator=gen, device="cuda").bfloat16()
    cache.append(k, v)
    want, want_l = cache.attend(q)
    cache.lens.zero_()
    cache.append(k, v * size.bfloat16())  # powers of two: the same codes
    o, lse = cache.attend(q)
    assert fa.fa_get_device_status() == 0
    # the scores are the same; each result is within 2^-8 |O| + (2^-11 + 2^-20 + n 2^-24) A of the exact one,
    # A <= max |v|, and 2^-8 of one result is 2^-8 (1 + 2^-7) of the other at most
    ratio = (o.float().unflatten(1, (Hkv, Hq)) / size[:, :, None]).flatten(1, 2)
    tol = 2.0 ** -7 * (1 + 2.0 ** -7) * want.float().abs() + 2 * (2.0 ** -11 + 2.0 ** -15) * float(v.abs().max())
    assert ((ratio - want.float()).abs() <= tol).all()
    assert float((lse - want_l).abs().max()) <= 2.0 ** -16
