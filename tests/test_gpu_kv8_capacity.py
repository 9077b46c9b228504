"""GPU tests of KV8Cache where a sequence cannot take what it is given: past its
capacity, counts out of range, lengths that the caller has set wrongly. Lengths
stay where nothing is written, and no output holds bytes that nobody wrote."""

import pytest

from attn_inputs import BASE_SEED
from kv8_util import ints

pytestmark = pytest.mark.gpu


def randn(gen, *shape):
    import torch
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def dirty(*shapes):
    """Fill the allocator's free blocks of these sizes with NaN bytes."""
    import torch
    held = [torch.full(s, 255, dtype=torch.uint8, device="cuda") for s in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("Nq", [1, 24])
@pytest.mark.parametrize("with_counts", [False, True])
def test_a_sequence_that_outgrows_its_pages_is_left_as_it_was(with_counts, Nq):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED)
    B, Hq, Hkv, d, cap = 3, 4, 2, 64, 64
    cache, other = (fa.KV8Cache(B, Hkv, d, cap, page=16) for _ in range(2))
    first = [cap - Nq + 1, 20, cap - Nq]  # the first sequence has no place for Nq more
    k, v = (randn(gen, B, Hkv, cap, d) for _ in range(2))
    for c in (cache, other):
        c.append(k, v, ints(*first))
    before = [t.clone() for t in (cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale)]
    k, v, q = randn(gen, B, Hkv, Nq, d), randn(gen, B, Hkv, Nq, d), randn(gen, B, Hq, Nq, d)
    other.append(k, v, ints(0, Nq, Nq))
    assert fa.fa_get_device_status() == 0
    cache.append(k, v, ints(Nq, Nq, Nq) if with_counts else None)
    assert fa.fa_get_device_status_detail()[:2] == (8, 31)
    assert cache.lens.tolist() == [first[0], 20 + Nq, cap]
    pages = cache.page_table[0].long()
    for t, was in zip((cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale), before):
        assert torch.equal(t[pages], was[pages])
    dirty((B, Hq, Nq, 2 * d), (B, Hq, Nq, 4))
    o, lse = cache.attend(q)
    want, want_l = other.attend(q)
    assert fa.fa_get_device_status() == 0
    assert torch.equal(o, want) and torch.equal(lse, want_l) and torch.isfinite(o).all()
    # and it goes on where it was: one token fits the first sequence, a second step none any more
    if Nq == 1:
        return
    cache.append(k[:, :, :1].contiguous(), v[:, :, :1].contiguous(), ints(1, 1, 0))
    assert fa.fa_get_device_status() == 0 and cache.lens.tolist() == [first[0] + 1, 21 + Nq, cap]


@pytest.mark.parametrize("bad", [-1, 6, 2 ** 31 - 1, -2 ** 31])
def test_counts_out_of_range_do_not_move_the_length(bad):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + 1)
    cache = fa.KV8Cache(2, 1, 64, 64, page=16)
    k = randn(gen, 2, 1, 5, 64)
    cache.append(k, k)
    cache.append(k, k, ints(bad, 3))
    assert fa.fa_get_device_status_detail()[:2] == (8, 31)
    assert cache.lens.tolist() == [5, 8]
    q = randn(gen, 2, 1, 5, 64)
    dirty((2, 1, 5, 128), (2, 1, 5, 4))
    o, lse = cache.attend(q, counts=ints(bad, 3))
    assert fa.fa_get_device_status_detail()[:2] == (8, 33)
    assert (o[0] == 0).all() and (lse[0] == 0).all() and torch.isfinite(o).all()


@pytest.mark.parametrize("Nq", [1, 40])
def test_lengths_set_out_of_range_give_rows_of_zeros(Nq):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + 2)
    cache = fa.KV8Cache(3, 1, 64, 64, page=16)
    k = randn(gen, 3, 1, 50, 64)
    cache.append(k, k)
    q = randn(gen, 3, 2, Nq, 64)
    want = cache.attend(q)
    assert fa.fa_get_device_status() == 0
    cache.lens.copy_(ints(65, 50, -3))
    dirty((3, 2, Nq, 128), (3, 2, Nq, 4))
    o, lse = cache.attend(q)
    assert fa.fa_get_device_status_detail()[:2] == (8, 33)
    assert (o[[0, 2]] == 0).all() and (lse[[0, 2]] == 0).all()
    assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])
    # nothing is written to them either
    cache.append(k[:, :, :1].contiguous(), k[:, :, :1].contiguous())
    assert fa.fa_get_device_status_detail()[:2] == (8, 31)
    assert cache.lens.tolist() == [65, 51, -3]


def test_a_captured_step_stops_at_the_capacity():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + 3)
    cache = fa.KV8Cache(2, 1, 64, 16, page=16)
    k, q = randn(gen, 2, 1, 1, 64), randn(gen, 2, 4, 1, 64)
    cache.append(randn(gen, 2, 1, 12, 64), randn(gen, 2, 1, 12, 64), ints(12, 5))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.append(k, k)
        o, lse = cache.attend(q)
    for step in range(1, 8):
        g.replay()
        torch.cuda.synchronize()
        assert cache.lens.tolist() == [min(16, 12 + step), 5 + step]
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        code = fa.fa_get_device_status_detail()[:2]
        assert code == ((8, 31) if step > 4 else (0, 0))


def test_a_call_refused_on_the_host_leaves_the_lengths():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + 4)
    cache = fa.KV8Cache(2, 2, 64, 64, page=16)
    k = randn(gen, 2, 2, 5, 64)
    cache.append(k, k)
    for bad, counts in ((k.float(), None), (k[..., :32], None), (k[:, :1], ints(1, 2)), (k, ints(1, 2).long()), (k, ints(1)),
                        (k, ints(1, 2).cpu())):
        with pytest.raises((TypeError, ValueError)):
            cache.append(bad, k, counts)
        assert cache.lens.tolist() == [5, 5]
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("B,Hq,Nq,d", [(B, *x) for B in (3, 70) for x in ((4, 1, 128), (2, 3, 256), (4, 40, 64), (2, 300, 128),
                                                                          (1, 200, 256))] +
                         [(2500, 4, 1, 128), (2500, 2, 3, 256), (2500, 4, 40, 64)])
def test_filled_rows(B, Hq, Nq, d):
    """Where there is a result it is fa_fwd_kv8's, bit for bit; everywhere else O = 0, L = 0."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + B + Nq)
    n = 320 if B <= 100 else 48
    cache = fa.KV8Cache(B, 1, d, n, page=32)
    cache.append(*(randn(gen, B, 1, n, d) for _ in range(2)))
    lens = torch.randint(0, n + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    counts = torch.randint(0, Nq + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    lens[0], counts[1], counts[2] = cache.page_table.shape[1] * 32 + 1, Nq + 1, 0
    q = randn(gen, B, Hq, Nq, d)
    ws = torch.empty(fa.fa_fwd_kv8_workspace_size(B, Hq, 1, Nq, d), dtype=torch.uint8, device="cuda")
    got = []
    for fn in (fa.fa_fwd_kv8, fa.fa_fwd_kv8_filled):
        o, lse = torch.full_like(q, 7.0), torch.full((B, Hq, Nq), 7.0, device="cuda")
        fn(q, *cache._cache()[:5], lens, o, lse, True, 0.1, counts, ws)
        assert fa.fa_get_device_status_detail()[:2] == (8, 33)
        got.append((o, lse))
    has = torch.arange(Nq, device="cuda")[None, :] < counts[:, None]
    has[0] = has[1] = False
    has = has[:, None].expand(B, Hq, Nq)
    (o, lse), (of, lf) = got
    assert (o[~has] == 7).all() and (lse[~has] == 7).all()
    assert (of[~has] == 0).all() and (lf[~has] == 0).all()
    assert torch.equal(o[has], of[has]) and torch.equal(lse[has], lf[has])
