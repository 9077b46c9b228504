"""Query rows past a sequence's count: what they hold is of no effect on the results,
not on their last bit (fa_fwd_kv8 of fa.h)."""

import pytest

from attn_inputs import BASE_SEED
from kv8_util import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Nq,d", [(2, 2, 64), (1, 4, 128), (4, 4, 128), (2, 4, 256), (1, 16, 64), (4, 10, 128), (2, 200, 64),
                                     (2, 100, 256)])
def test_rows_past_the_count_do_not_show_in_the_others(Hq, Nq, d):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + Nq + d)
    B, Hkv, n = 12, 2, 600
    cache = fa.KV8Cache(B, Hkv, d, n, page=16)
    cache.append(*(torch.randn(B, Hkv, n, d, generator=gen, device="cuda").bfloat16() for _ in range(2)))
    counts = ints(*(max(1, (Nq * (b + 1)) // (B + 1)) for b in range(B)))
    q = (3 * torch.randn(B, Hkv * Hq, Nq, d, generator=gen, device="cuda")).bfloat16()  # references move often
    past = (torch.arange(Nq, device="cuda")[None, :] >= counts[:, None])[:, None, :, None].expand_as(q)
    first = None
    for fill in (0.0, 1.0, -300.0, 3e38, float("inf"), float("nan")):
        x = torch.where(past, torch.full_like(q, fill), q)
        o, lse = cache.attend(x.contiguous(), counts=counts)
        assert fa.fa_get_device_status() == 0
        if first is None:
            first = o, lse
            assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), fill
