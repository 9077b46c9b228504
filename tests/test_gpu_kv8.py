"""GPU parity of the paged 8-bit cache: fa_kv8_append byte for byte and
fa_kv8_gather bit for bit against the float64 oracle. Scales are powers of two,
so every step before the one rounding to e4m3 is exact and nothing is left to a
tolerance."""

import numpy as np
import pytest

from attn_inputs import BASE_SEED, bf16_bits_to_f64, f32_to_bf16_bits
from gpu_util import to_device, to_host64
from kv8_util import Pools, ints
from oracle import cache_ops as co

pytestmark = pytest.mark.gpu


def values(rng, *shape, spread=0.0):
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, shape[:2] + (1, 1)))
    bits = f32_to_bf16_bits(x.astype(np.float32))
    return bits, bf16_bits_to_f64(bits)


def append(p, kb, vb, lens, counts):
    import exact_softmax_attention_fa_gb300 as fa
    c = None if counts is None else ints(*counts)
    fa.fa_kv8_append(to_device(kb), to_device(vb), *p.device(), ints(*lens), c)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_is_the_oracle_byte_for_byte(d, page):
    B, Hkv = 3, 2
    p = Pools(B, Hkv, d, page, 5, BASE_SEED + page + d)
    lens = [0] * B
    # ragged pieces: whole pages, a piece that ends inside a page, single tokens with a growing spread
    for n, counts, spread in ((page * 2 + 3, [page * 2 + 3, 1, page], 0.0), (1, [1, 1, 1], 3.0), (5, [0, 5, 2], 6.0),
                              (page, [page, page - 1, page], 1.0), (1, [1, 0, 1], 9.0)):
        (kb, k), (vb, v) = (values(p.rng, B, Hkv, n, d, spread=spread) for _ in range(2))
        lens = [a + c for a, c in zip(lens, counts)]
        append(p, kb, vb, lens, counts)
        p.fill(k, v, lens, counts)
        assert p.same(), (n, counts)
    import exact_softmax_attention_fa_gb300 as fa
    assert fa.fa_get_device_status() == 0


def test_append_without_counts_and_empty_calls():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    p = Pools(2, 1, 64, 16, 3, BASE_SEED + 1)
    (kb, k), (vb, v) = (values(p.rng, 2, 1, 20, 64) for _ in range(2))
    append(p, kb, vb, [20, 33], None)  # the second sequence starts at 13, in the middle of a page
    p.fill(k, v, [20, 33], [20, 20])
    assert p.same()
    append(p, kb, vb, [20, 33], [0, 0])
    z = torch.empty(2, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    fa.fa_kv8_append(z, z, *p.device(), ints(20, 33))
    assert p.same() and fa.fa_get_device_status() == 0


def test_append_of_zeros_extremes_and_values_that_are_not_finite():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    p = Pools(1, 2, 64, 16, 4, BASE_SEED + 2)
    x = np.zeros((1, 2, 64, 64), np.float32)
    x[0, 0, 16:32] = 3e38 * np.linspace(-1, 1, 64)      # the largest bf16 values
    x[0, 0, 32:48] = 2.0 ** -130                        # subnormal bf16
    x[0, 1, 0, :4] = [np.nan, np.inf, -np.inf, 1.0]     # the scale comes from the finite ones
    x[0, 1, 16:32] = np.inf                             # a page without a finite value
    x[0, 1, 32:48] = 448.0
    x[0, 1, 48:] = 448.0 * 1.01
    t = torch.from_numpy(x).to("cuda", torch.bfloat16)
    fa.fa_kv8_append(t, t, *p.device(), ints(64))
    f = to_host64(t)
    p.fill(f, f, [64], [64])
    assert p.same() and fa.fa_get_device_status() == 0
    assert (p.scale[0][p.table[0], 1] == [2.0 ** -8, 2.0 ** -100, 1.0, 2.0]).all()


def test_a_growing_scale_moves_the_codes_before_it():
    p = Pools(1, 1, 64, 16, 1, BASE_SEED + 3)
    for i in range(16):
        (kb, k), (vb, v) = (values(p.rng, 1, 1, 1, 64) for _ in range(2))
        m = np.float32(2.0 ** (1.7 * i - 9))
        kb, vb = (f32_to_bf16_bits(x.astype(np.float32) * m) for x in (k, v))
        k, v = bf16_bits_to_f64(kb), bf16_bits_to_f64(vb)
        append(p, kb, vb, [i + 1], None)
        p.fill(k, v, [i + 1], [1])
        assert p.same(), i


def test_append_refuses_bad_lengths_and_pages_and_writes_nothing_there():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    B, Hkv, d, page = 6, 1, 64, 16
    p = Pools(B, Hkv, d, page, 2, BASE_SEED + 4)
    (kb, k), (vb, v) = (values(p.rng, B, Hkv, 4, d) for _ in range(2))
    pool = len(p.code[0])
    p.d_table[4, 0] = pool
    p.d_table[5, 1] = -1
    # too many new tokens; more than there are; a negative count; more than the pages hold; pages outside the pool
    append(p, kb, vb, [30, 2, 8, 33, 4, 18], [5, 3, -1, 4, 4, 4])
    assert fa.fa_get_device_status_detail()[:2] == (8, 31)
    # only the part of sequence 5 that lies in its first page is written
    c = [k[5:, :, :2], v[5:, :, :2]]
    for i in range(2):
        p.code[i], p.scale[i] = co.cache_append(c[i], p.code[i], p.scale[i], p.table[5:], [16], [2])
    assert p.same()
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_gather_is_exact_and_leaves_later_rows(d, page):
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    B, Hkv, n = 4, 3, 150
    mp = -(-170 // page)
    p = Pools(B, Hkv, d, page, mp, BASE_SEED + 5 + page)
    lens = [170, 0, 1, 149]
    (_, k), (_, v) = (values(p.rng, B, Hkv, 170, d) for _ in range(2))
    p.fill(k, v, lens, lens)
    p.upload()
    # entries past a sequence's last page are not read
    for b in range(B):
        p.d_table[b, -(-lens[b] // page):] = -1
    out = [torch.full((B, Hkv, n, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.fa_kv8_gather(*p.device(), ints(*lens), *out)
    assert fa.fa_get_device_status() == 0
    for i in range(2):
        got = to_host64(out[i])
        for b in range(B):
            m = min(lens[b], n)
            want = co.cache_rows(p.code[i], p.scale[i], p.table[b], m)
            assert np.array_equal(got[b, :, :m], want)
            assert (got[b, :, m:] == 5.0).all()


def test_gather_refuses_bad_lengths_and_pages():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    p = Pools(3, 1, 64, 16, 2, BASE_SEED + 6)
    (_, k), (_, v) = (values(p.rng, 3, 1, 32, 64) for _ in range(2))
    p.fill(k, v, [32] * 3, [32] * 3)
    p.upload()
    p.d_table[2, 0] = 1 << 30
    out = [torch.full((3, 1, 32, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.fa_kv8_gather(*p.device(), ints(33, -1, 32), *out)
    assert fa.fa_get_device_status_detail()[:2] == (8, 32)
    for i in range(2):
        got = to_host64(out[i])
        assert (got[:2] == 5.0).all() and (got[2, :, :16] == 5.0).all()
        assert np.array_equal(got[2, :, 16:], co.cache_rows(p.code[i], p.scale[i], p.table[2], 32)[:, 16:])


def test_pools_past_32_bit_offsets():
    """Pages whose byte offsets are above 2^32 (the pool holds 5 GB of codes)."""
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    page, Hkv, d = 128, 8, 256
    pages = (5 << 30) // (page * Hkv * d)
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    ks, vs = (torch.empty(pages, Hkv, device="cuda") for _ in range(2))
    table = ints(pages - 1, 0).view(1, 2)
    x = torch.randn(1, Hkv, 200, d, device="cuda").bfloat16()
    y = torch.randn(1, Hkv, 200, d, device="cuda").bfloat16()
    fa.fa_kv8_append(x, y, kc, vc, ks, vs, table, ints(200))
    a, b = torch.empty_like(x), torch.empty_like(y)
    fa.fa_kv8_gather(kc, vc, ks, vs, table, ints(200), a, b)
    assert fa.fa_get_device_status() == 0
    for got, want, s in ((a, x, ks), (b, y, vs)):
        step = s[table[0].long()].max()
        assert ((got.float() - want.float()).abs() <= 2.0 ** -4 * want.float().abs() + 2.0 ** -10 * step).all()


def test_append_and_gather_replay_from_a_graph_with_new_lengths():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    B, Hkv, d, page = 2, 2, 128, 32
    p = Pools(B, Hkv, d, page, 3, BASE_SEED + 7)
    k, v = (torch.zeros(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = ints(0, 40)
    out = [torch.zeros(B, Hkv, 96, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    (_, k0), (_, v0) = (values(p.rng, B, Hkv, 40, d) for _ in range(2))
    p.fill(k0, v0, [0, 40], [0, 40])
    p.upload()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        lens.add_(1)
        fa.fa_kv8_append(k, v, *p.device(), lens)
        fa.fa_kv8_gather(*p.device(), lens, *out)
    for i in range(5):
        (kb, kf), (vb, vf) = (values(p.rng, B, Hkv, 1, d, spread=4.0) for _ in range(2))
        k.copy_(to_device(kb))
        v.copy_(to_device(vb))
        g.replay()
        torch.cuda.synchronize()
        p.fill(kf, vf, [i + 1, 41 + i], [1, 1])
        assert p.same()
        for j in range(2):
            for b, n in enumerate((i + 1, 41 + i)):
                assert np.array_equal(to_host64(out[j][b])[:, :n], co.cache_rows(p.code[j], p.scale[j], p.table[b], n))
    assert fa.fa_get_device_status() == 0


def test_tensors_are_checked():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    p = Pools(1, 1, 64, 16, 1, BASE_SEED + 8)
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    dev = p.device()
    for bad, exc in ((dict(k=x.float()), TypeError), (dict(k=x[..., :32]), ValueError), (dict(lens=ints(1).long()), ValueError),
                     (dict(lens=ints(1, 1)), ValueError), (dict(lens=ints(1).cpu()), ValueError)):
        with pytest.raises(exc):
            fa.fa_kv8_append(bad.get("k", x), x, *dev, bad.get("lens", ints(1)))
    with pytest.raises(TypeError):
        fa.fa_kv8_append(x, x, dev[0].to(torch.int8), *dev[1:], ints(1))
    with pytest.raises(ValueError):
        fa.fa_kv8_append(x, x, dev[0], dev[1][:1], *dev[2:], ints(1))
    assert fa.fa_get_device_status() == 0
