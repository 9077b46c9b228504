"""The attention over the 8-bit cache against the dense attention on the gathered cache
(append, read-back and both attentions together), and how exactly queries are held."""

import numpy as np
import pytest

from attn_inputs import BASE_SEED
from kv8_util import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(8, 2, 1), (8, 8, 1), (8, 2, 30), (8, 2, 200)])
def test_relative_difference_from_the_dense_attention(Hq, Hkv, Nq, d, page, causal):
    """V has random signs, so |O|^2 is sum p^2 v^2 on average. The dense kernel's weights are rounded to bf16, at most
    2^-8 of each and of either sign: 2^-8 / sqrt(3) of |O| in the mean square; both outputs are, again 2^-8 / sqrt(3)
    each; everything else is below 2^-11. Together 2^-8 of the norm; 2^-7 is allowed. One group of 16 of the
    1000 keys left out would be sqrt(16 / 1000) = 2^-3 of it."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + d + Nq)
    B, n = 3, 1000
    mp = -(-n // page)
    table = torch.randperm(B * mp + 5, generator=gen, device="cuda")[:B * mp].view(B, mp).to(torch.int32)
    cache = fa.KV8Cache(B, Hkv, d, n, page=page, page_table=table, num_pages=B * mp + 5)
    k, v = (torch.randn(B, Hkv, n, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, Nq, d, generator=gen, device="cuda").bfloat16()
    for lo, hi in ((0, 313), (313, 314), (314, n)):
        cache.append(k[:, :, lo:hi].contiguous(), v[:, :, lo:hi].contiguous())
    kk, vv = cache.gather(n)
    # the cache itself: half a step of e4m3, at most twice where a page's scale grew, or of its smallest step
    assert float(((kk - k).float().norm() / k.float().norm())) <= 2.0 ** -4
    ref, ref_l = torch.empty_like(q), torch.empty(B, Hq, Nq, device="cuda")
    fa.fa_fwd_splitkv(q, kk, vv, ref, ref_l, causal, fa.default_scale(d), 1)
    o, lse = cache.attend(q, causal=causal)
    assert fa.fa_get_device_status() == 0
    diff, norm = (o.float() - ref.float()).double().square().sum((2, 3)), ref.double().square().sum((2, 3))
    assert float((diff / norm).sqrt().max()) <= 2.0 ** -7  # of every head for itself: at least d elements
    # both: sums of d products and of n weights in fp32
    assert float((lse - ref_l).abs().max()) <= 2.0 ** -10


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,top,e", [(1, 7, 2.0 ** -21), (16, 7, 2.0 ** -21), (40, 3, 2.0 ** -17), (300, 3, 2.0 ** -17)])
def test_the_smallest_columns_of_a_query_are_held_to_a_fraction_of_its_largest(rows, top, e, d):
    """A row of 128 and 2^-top + 2^-(top + 7), the worst place between two steps of its pieces: the score is off by at
    most e of the largest times the key, and by half of that at least (the bound is met, not only kept)."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    if d == 256 and rows == 16:
        rows = 8  # more take the other kernel
    q = torch.zeros(1, 1, rows, d, device="cuda")
    q[..., 0] = 128.0
    q[..., 5] = 2.0 ** -top + 2.0 ** -(top + 7)
    cache = fa.KV8Cache(1, 1, d, 16, page=16)
    k = torch.zeros(1, 1, 1, d, device="cuda")
    k[..., 5] = 448.0
    cache.append(k.bfloat16(), k.bfloat16())
    scale = 2.0 ** -6
    q16 = q.bfloat16()
    assert torch.equal(q16.float(), q)
    _, lse = cache.attend(q16, causal=False, scale=scale)
    assert fa.fa_get_device_status() == 0
    err = (lse.double() - scale * 448.0 * float(q[0, 0, 0, 5])).abs()
    # one key: L is its score; ln 2 * log2(e) and the exponent's rounding: 4 steps of 2^-24 of it
    rest = 2.0 ** -22 * float(lse.abs().max())
    assert float(err.max()) <= scale * 448.0 * 128.0 * e + rest
    if rows > 16:
        assert float(err.min()) >= scale * 448.0 * 128.0 * e / 2 - rest
