"""GPU parity of the attention over the paged 8-bit cache (fa_fwd_kv8) against
the float64 oracle on the same codes and scales.

Tolerances. With p the exact weights, A = sum_j p_j |v_j| per output column and
n keys: a weight is rounded to fp16, half a step or 2^-11 of itself, and its
pieces hold that exactly or to 2^-24 of the row's largest weight; exp2 is within 2^-22, n terms are summed in fp32 in runs of 16 (at most n 2^-24). A
score is a sum of d exact products in fp32 by the tensor core (two units of 2^-23
for each of d / 16 steps, and four for its scaling) of query values that are
exact or within e max|q|: e = 2^-22 up to 16 rows per K/V head (8 at d = 256), whose two e4m3
pieces are summed apart with a factor of 2^4 between them, and 2^-18 above,
where they are not. So it is off by at most
  delta = scale max_j ((d/16 + 4) 2^-22 sum |q k_j| + e max|q| sum |k_j|),
which moves every weight by at most 2 delta. So
  |O - O_ref| <= 2^-8 |O_ref| + A (2^-11 + 2^-20 + n 2^-24 + 2 delta)
                 + 2^-24 max(p) sum_j |v_j|
  |L - L_ref| <= delta + 2^-20 + n 2^-24 + 2^-21 |L_ref|.
"""

import types

import numpy as np
import pytest

from attn_inputs import BASE_SEED, bf16_bits_to_f64, f32_to_bf16_bits
from gpu_util import scale_f32, to_device, to_host64
from kv8_util import Pools, ints
from oracle import cache_ops as co

pytestmark = pytest.mark.gpu

MARK = 5.0


def bf16(rng, *shape, spread=1.0):
    bits = f32_to_bf16_bits((rng.standard_normal(shape) * spread).astype(np.float32))
    return bits, bf16_bits_to_f64(bits)


def filled(B, Hkv, d, page, lens, seed, mult=None):
    """A device cache that holds lens[b] tokens, its host copy, and the table
    with entries past each sequence's last page set to -1 on the device."""
    p = Pools(B, Hkv, d, page, max(1, -(-max(lens) // page)), seed)
    n = max(1, max(lens))
    (_, k), (_, v) = (bf16(p.rng, B, Hkv, n, d) for _ in range(2))
    if mult is not None:
        v = v * mult(n)[:, None]
    p.fill(k, v, lens, lens)
    p.upload()
    for b in range(B):
        p.d_table[b, -(-lens[b] // page):] = -1
    return p


def call(p, qb, lens, counts, causal, scale, stream=None):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    q = to_device(qb)
    B, Hq, Nq, d = q.shape
    o = torch.full_like(q, MARK)
    lse = torch.full((B, Hq, Nq), MARK, device="cuda")
    ws = torch.full((fa.fa_fwd_kv8_workspace_size(B, Hq, p.code[0].shape[1], Nq, d),), 255, dtype=torch.uint8,
                    device="cuda")
    fa.fa_fwd_kv8(q, *p.device(), ints(*lens), o, lse, causal, scale, None if counts is None else ints(*counts), ws,
                  stream)
    return o, lse


def compare(p, q, lens, counts, causal, scale, o, lse, table=None):
    """Check every row of every sequence against the definition."""
    B, Hq, Nq, d = q.shape
    Hkv = p.code[0].shape[1]
    e_q = 2.0 ** -22 if Hq // Hkv * Nq <= (8 if d == 256 else 16) else 2.0 ** -18
    o, lse = to_host64(o), lse.double().cpu().numpy()
    for b in range(B):
        n, c = lens[b], Nq if counts is None else counts[b]
        assert (o[b, :, c:] == MARK).all() and (lse[b, :, c:] == MARK).all()
        k = co.cache_rows(p.code[0], p.scale[0], p.table[b], n)
        v = co.cache_rows(p.code[1], p.scale[1], p.table[b], n)
        see = np.arange(n)[None, :] < (np.minimum(n, n - c + 1 + np.arange(c)) if causal else np.full(c, n))[:, None]
        for h in range(Hq):
            kh, vh = k[h // (Hq // Hkv)], v[h // (Hq // Hkv)]
            t = np.where(see, scale * (q[b, h, :c] @ kh.T), -np.inf)
            aq, ak = np.abs(q[b, h, :c]), np.abs(kh)
            mag = scale * ((d / 16 + 4) * 2.0 ** -22 * (aq @ ak.T) +
                           e_q * aq.max(1, initial=0)[:, None] * ak.sum(1)[None, :])
            delta = np.max(np.where(see, mag, 0), axis=1, initial=0)
            any_ = see.any(1)
            top = np.max(t, axis=1, initial=-np.inf, where=see)
            e = np.exp(t - np.where(any_, top, 0)[:, None])
            l = e.sum(1)
            w = e / np.where(any_, l, 1)[:, None]
            with np.errstate(divide="ignore"):
                l_ref = np.where(any_, top + np.log(l), -np.inf)
            o_ref, A = w @ vh, w @ np.abs(vh)
            assert (lse[b, h, :c][~any_] == -np.inf).all() and (o[b, h, :c][~any_] == 0).all()
            err = np.abs(o[b, h, :c] - o_ref)
            tol = 2.0 ** -8 * np.abs(o_ref) + A * (2.0 ** -11 + 2.0 ** -20 + n * 2.0 ** -24 + 2 * delta[:, None])
            tol += 2.0 ** -24 * w.max(1, initial=0)[:, None] * (see @ np.abs(vh))
            assert (err <= tol).all(), (b, h, err.max(), (err - tol).max())
            e_l = np.abs(lse[b, h, :c][any_] - l_ref[any_])
            assert (e_l <= delta[any_] + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -21 * np.abs(l_ref[any_])).all(), (b, h)


def check(B, Hq, Hkv, Nq, d, page, lens, counts, causal, seed, mult=None):
    import exact_softmax_attention_fa_gb300 as fa
    p = filled(B, Hkv, d, page, lens, seed, mult)
    qb, q = bf16(p.rng, B, Hq, Nq, d)
    scale = scale_f32(d)
    o, lse = call(p, qb, lens, counts, causal, scale)
    assert fa.fa_get_device_status() == 0
    compare(p, q, lens, counts, causal, scale, o, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (4, 1), (6, 2), (16, 2), (16, 1), (20, 1)])
def test_decode(d, page, Hq, Hkv):
    # one query each, sequences that end at, before and behind the edges of steps and pages, one without tokens
    lens = [1, 15, 16, 17, 0, 127, 128, 129, 300]
    check(len(lens), Hq, Hkv, 1, d, page, lens, [1, 1, 1, 1, 0, 1, 1, 1, 1], True, BASE_SEED + page + d + Hq)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 1, 2), (3, 1, 5), (4, 2, 16), (2, 2, 33), (8, 1, 40), (2, 1, 130)])
def test_blocks_of_new_tokens(d, causal, Hq, Hkv, Nq):
    lens = [Nq, Nq + 1, 200 + Nq, 7, 0]
    counts = [Nq, max(1, Nq - 1), Nq, min(Nq, 7), 0]
    check(len(lens), Hq, Hkv, Nq, d, 32, lens, counts, causal, BASE_SEED + Nq + d)


@pytest.mark.parametrize("causal", [False, True])
def test_rows_that_see_no_key(causal):
    # more queries than tokens: the first stand before the sequence; a sequence without tokens
    check(3, 4, 2, 6, 64, 16, [3, 0, 20], [6, 4, 6], causal, BASE_SEED + 11)
    check(3, 4, 2, 40, 64, 16, [3, 0, 50], [40, 4, 33], causal, BASE_SEED + 11)


@pytest.mark.parametrize("B", [33, 70])
def test_many_ragged_sequences(B):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 90, B)]
    lens[0] = lens[-1] = 0
    check(B, 4, 2, 1, 64, 16, lens, [min(1, x) for x in lens], True, BASE_SEED + B)


@pytest.mark.parametrize("d,page,Hq,Nq", [(128, 64, 4, 1), (64, 16, 8, 2), (256, 32, 2, 1), (128, 16, 2, 70)])
def test_long_caches_shared_by_many_warps(d, page, Hq, Nq):
    check(2, Hq, 1, Nq, d, page, [9001, 4500], [Nq, Nq], True, BASE_SEED + d + page)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,page,Hq,Hkv,Nq,lens", [
    (128, 64, 6, 2, 17, [5000, 130, 0]),    # 51 rows: one tile of rows, runs of an odd and an even number of key tiles
    (64, 16, 4, 4, 97, [2049, 1, 1300]),    # 97 rows
    (128, 128, 5, 1, 60, [4100, 300, 77]),  # 300 rows: two blocks, positions shared between tiles
    (64, 32, 2, 2, 300, [3333, 300]),       # 300 rows of one head
    (256, 32, 3, 1, 100, [3000, 700]),      # 300 rows, one tile a block
])
def test_chunks_shared_by_many_blocks(causal, d, page, Hq, Hkv, Nq, lens):
    counts = [min(Nq, n) for n in lens]
    counts[1] = min(counts[1], 5)
    check(len(lens), Hq, Hkv, Nq, d, page, lens, counts, causal, BASE_SEED + d + Nq)


@pytest.mark.parametrize("Nq", [33, 90])
def test_chunks_of_many_ragged_sequences(Nq):
    rng = np.random.default_rng(Nq)
    lens = [int(x) for x in rng.integers(0, 400, 40)]
    lens[0] = lens[-1] = 0
    counts = [int(rng.integers(0, min(Nq, n) + 1)) for n in lens]
    check(40, 4, 2, Nq, 64, 16, lens, counts, True, BASE_SEED + Nq)


@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_values_whose_scales_differ_by_powers_of_two(d, Nq):
    # pages of values from 2^-40 to 2^40 of one another, in rising, falling and mixed order
    for k, mult in enumerate((lambda n: np.exp2(np.arange(n) // 16 * 4.0 - 40), lambda n: np.exp2(40 - np.arange(n) // 16 * 4.0),
                              lambda n: np.exp2((np.arange(n) // 16 * 7) % 11 * 8.0 - 40))):
        check(1, 4, 2, Nq, d, 16, [330], [Nq], True, BASE_SEED + 20 + k, mult)


@pytest.mark.parametrize("Nq", [1, 40])
def test_zero_values_and_zero_queries(Nq):
    import exact_softmax_attention_fa_gb300 as fa
    p = filled(1, 1, 64, 16, [2000], BASE_SEED + 30, lambda n: np.zeros(n))
    qb, q = bf16(p.rng, 1, 8, Nq, 64)
    qb[0, 4:], q[0, 4:] = 0, 0
    o, lse = call(p, qb, [2000], None, False, 0.125)
    assert fa.fa_get_device_status() == 0
    assert (o == 0).all()
    compare(p, q, [2000], None, False, 0.125, o, lse)


@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 12])
def test_query_sizes(Nq, size):
    import exact_softmax_attention_fa_gb300 as fa
    p = filled(2, 2, 128, 32, [500, 77], BASE_SEED + 31)
    qb, q = bf16(p.rng, 2, 4, Nq, 128, spread=size)
    scale = float(np.float32(0.09 / size))
    o, lse = call(p, qb, [500, 77], None, True, scale)
    assert fa.fa_get_device_status() == 0
    compare(p, q, [500, 77], None, True, scale, o, lse)


@pytest.mark.parametrize("Nq", [1, 40])
def test_peaked_scores(Nq):
    # large scores: the reference keeps moving, and most weights are 0
    import exact_softmax_attention_fa_gb300 as fa
    p = filled(1, 1, 64, 64, [1500], BASE_SEED + 32)
    qb, q = bf16(p.rng, 1, 8, Nq, 64, spread=8.0)
    o, lse = call(p, qb, [1500], None, True, 0.125)
    assert fa.fa_get_device_status() == 0
    compare(p, q, [1500], None, True, 0.125, o, lse)


@pytest.mark.parametrize("Nq", [1, 40])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(Nq):
    import exact_softmax_attention_fa_gb300 as fa
    lens = [100, 100, 100]
    p = filled(3, 1, 64, 16, lens, BASE_SEED + 33)
    p.code[0][p.table[0, 1], 0, 3, 5] = 0x7F    # a key of sequence 0
    p.code[1][p.table[1, 2], 0, 4, 6] = 0xFF    # a value of sequence 1
    p.upload()
    qb, q = bf16(p.rng, 3, 4, Nq, 64)
    o, lse = call(p, qb, lens, None, True, 0.125)
    assert fa.fa_get_device_status() == 0
    assert o[0].isnan().all() and lse[0].isnan().all()
    assert o[1, ..., 6].isnan().all() and not o[1, ..., :6].isnan().any() and not lse[1].isnan().any()
    assert not o[2].isnan().any()
    # a query that is not finite spoils its own row alone
    qb[2, 1, 0, 3] = 0x7FC0
    o2, lse2 = call(p, qb, lens, None, True, 0.125)
    import torch
    assert o2[2, 1, 0].isnan().all()
    keep = torch.ones(4, Nq, dtype=torch.bool, device="cuda")
    keep[1, 0] = False
    assert torch.equal(o2[2][keep], o[2][keep]) and torch.equal(lse2[2][keep], lse[2][keep])


@pytest.mark.parametrize("Nq", [1, 40])
def test_bad_lengths_counts_and_pages(Nq):
    import exact_softmax_attention_fa_gb300 as fa
    lens = [100, 100, 100, 100]
    p = filled(4, 1, 64, 16, lens, BASE_SEED + 34)
    qb, q = bf16(p.rng, 4, 4, Nq, 64)
    bad = [100, 113, -1, 100]
    o, lse = call(p, qb, bad, [Nq, Nq, 0, Nq + 1], True, 0.125)
    assert fa.fa_get_device_status_detail()[:2] == (8, 33)
    assert (o[1:] == MARK).all() and (lse[1:] == MARK).all()
    good, good_l = call(p, qb, lens, None, True, 0.125)
    assert fa.fa_get_device_status() == 0
    compare(p, q, lens, None, True, 0.125, good, good_l)
    # tokens on a page outside the pool are not seen: the same as a sequence without that page
    p.d_table[3, 2] = len(p.code[0])
    o, lse = call(p, qb, lens, None, False, 0.125)
    assert fa.fa_get_device_status_detail()[:2] == (8, 33)
    keep = [0, 1, 3, 4, 5, 6]
    short = types.SimpleNamespace(code=p.code, scale=p.scale, table=p.table[3:, keep])
    compare(short, q[3:], [84], None, False, 0.125, o[3:], lse[3:])
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("Nq", [1, 3, 40])
def test_results_do_not_depend_on_timing_streams_or_the_workspace(Nq):
    import torch
    p = filled(3, 2, 128, 64, [5000, 1, 2600], BASE_SEED + 35)
    qb, _ = bf16(p.rng, 3, 8, Nq, 128)
    first = call(p, qb, [5000, 1, 2600], [Nq, 1, Nq], True, 0.09)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [call(p, qb, [5000, 1, 2600], [Nq, 1, Nq], True, 0.09) for _ in range(2)]
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(call(p, qb, [5000, 1, 2600], [Nq, 1, Nq], True, 0.09))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_agrees_with_the_dense_attention_on_the_gathered_cache():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, Nq, n, d = 2, 8, 2, 64, 1000, 128
    cache = fa.KV8Cache(B, Hkv, d, n, page=64)
    k, v = (torch.randn(B, Hkv, n, d, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, Nq, d, device="cuda").bfloat16()
    cache.append(k, v)
    kk, vv = cache.gather(n)
    ref = torch.empty_like(q), torch.empty(B, Hq, Nq, device="cuda")
    fa.fa_fwd_splitkv(q, kk, vv, *ref, True, fa.default_scale(d), 1)
    o, lse = cache.attend(q)
    assert fa.fa_get_device_status() == 0
    # the dense kernel rounds its weights to bf16: 2^-8 of them more
    A = float(vv.abs().max())
    assert float((o.float() - ref[0].float()).abs().max()) <= 2 * 2.0 ** -8 * A
    assert float((lse - ref[1]).abs().max()) <= 1e-3


@pytest.mark.parametrize("captured", [False, True])
def test_a_decoding_loop_from_projection_to_output(captured):
    """prompt, then single tokens: norm + rotation -> append -> attention, each step
    checked against the oracle on what the cache holds; replayed from a graph
    whose lengths and positions move on the device."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, d, page = 2, 4, 2, 64, 16
    prompt = [20, 33]
    cos, sin = fa.rope_tables(128, d)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    host = Pools(B, Hkv, d, page, 4, BASE_SEED + 40, spare=0)
    host.table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)
    cache = fa.KV8Cache(B, Hkv, d, 64, page)
    H = Hq + 2 * Hkv
    x = torch.randn(B, 33, H, d, device="cuda").bfloat16()
    qi, ki, vi = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], dim=2))
    counts = ints(*prompt)
    pos = torch.arange(33, dtype=torch.int32, device="cuda").repeat(B, 1).contiguous()
    q, k, v = fa.norm_rope(qi, ki, vi, w, w, cos, sin, pos)
    cache.append(k, v, counts)
    o, lse = cache.attend(q, counts=counts)
    lens = list(prompt)
    host.fill(to_host64(k), to_host64(v), lens, prompt)

    def step_check(q, o, lse, c):
        host.d_code, host.d_scale = (cache.k_cache, cache.v_cache), (cache.k_scale, cache.v_scale)
        used = [host.table[b, i] for b in range(B) for i in range(-(-lens[b] // page))]
        for i in range(2):
            assert np.array_equal(host.d_scale[i].cpu().numpy()[used], host.scale[i][used])
        o2, l2 = o.clone(), lse.clone()
        for b in range(B):
            assert (o2[b, :, c[b]:] == 0).all()
            o2[b, :, c[b]:], l2[b, :, c[b]:] = MARK, MARK
        compare(host, to_host64(q), lens, c, True, fa.default_scale(d), o2, l2)

    step_check(q, o, lse, prompt)
    x1 = torch.zeros(B, 1, H, d, dtype=torch.bfloat16, device="cuda")
    q1, k1, v1 = (t.transpose(1, 2) for t in x1.split([Hq, Hkv, Hkv], dim=2))

    def step():
        p1 = cache.lens.view(B, 1).clone()  # the new token's position
        q, k, v = fa.norm_rope(q1, k1, v1, w, w, cos, sin, p1)
        cache.append(k, v)
        return q, k, v, *cache.attend(q)

    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
    for _ in range(6):
        x1.copy_(torch.randn(B, 1, H, d, device="cuda"))
        if captured:
            graph.replay()
            q, k, v, o, lse = held
        else:
            q, k, v, o, lse = step()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        host.fill(to_host64(k), to_host64(v), lens, [1] * B)
        step_check(q, o, lse, [1] * B)
    assert cache.lens.tolist() == lens and fa.fa_get_device_status() == 0


def test_two_graphs_at_the_same_time():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    B, Hq, Hkv, d, n = 2, 8, 2, 128, 3000
    graphs, outs, want = [], [], []
    cache = fa.KV8Cache(B, Hkv, d, n)
    cache.append(*(torch.randn(B, Hkv, n, d, device="cuda").bfloat16() for _ in range(2)))
    qs = [torch.randn(B, Hq, 1, d, device="cuda").bfloat16() for _ in range(2)]
    for q in qs:
        want.append(cache.attend(q))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cache.attend(q))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tensors_are_checked():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    c = fa.KV8Cache(1, 2, 64, 32, 16)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 4, 1, device="cuda")
    with pytest.raises(TypeError):
        c.attend(q.half())
    with pytest.raises(ValueError):
        c.attend(q[:, :3])
    with pytest.raises(ValueError):
        c.attend(torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        fa.fa_fwd_kv8(q, *c._cache(), o, lse.half(), True, 0.1)
    with pytest.raises(fa.FAError) as e:
        fa.fa_fwd_kv8(q, *c._cache(), o, lse, True, 0.1)  # no workspace
    assert e.value.status == 4
    with pytest.raises(fa.FAError) as e:
        c.attend(q, scale=float("nan"))
    assert e.value.status == 1
    assert c.attend(torch.empty(1, 4, 0, 64, dtype=torch.bfloat16, device="cuda"))[0].shape == (1, 4, 0, 64)
    assert fa.fa_get_device_status() == 0


def test_workspaces_are_one_run_of_bytes():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    c = fa.KV8Cache(1, 2, 64, 32, 16)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 4, 1, device="cuda")
    size = fa.fa_fwd_kv8_workspace_size(1, 4, 2, 1, 64)
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for ws in (one.expand(size), torch.zeros(2 * size, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            fa.fa_fwd_kv8(q, *c._cache(), o, lse, True, 0.125, None, ws)
    k = q[:, :2].contiguous()
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        fa.norm_rope_backward(q, k, None, q, k, w, w, workspace=one.expand(1 << 20))
    assert fa.fa_get_device_status() == 0


def test_the_chain_on_a_stream_of_its_own_while_others_allocate():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED)
    B, Hq, Hkv, N, d = 2, 8, 2, 700, 128
    x = torch.randn(B, Hq + 2 * Hkv, N, d, generator=gen, device="cuda").bfloat16()
    wq, wk = (torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    cos, sin = fa.rope_tables(N, d)
    xq, xk, xv = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    caches = []  # made on the current stream, so they stay until the side stream is done

    def chain(stream):
        q, k, v = fa.norm_rope(xq, xk, xv, wq, wk, cos, sin, stream=stream)
        cache = fa.KV8Cache(B, Hkv, d, N)
        caches.append(cache)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        cache.append(k, v, stream=stream)
        o, lse = cache.attend(q, stream=stream)
        return (o, lse, *fa.norm_rope_backward(o, k, v, xq, xk, wq, wk, cos, sin, stream=stream))

    want = chain(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    runs = []
    for _ in range(8):
        runs.append(chain(side))
        for size in (1 << 20, 1 << 22):  # what the chain has freed is not handed out here
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    side.synchronize()
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("Hq,Nq,d", [(4, 20, 128), (4, 80, 128), (2, 40, 64), (2, 40, 256)])
@pytest.mark.parametrize("role", [41, 42, 43, 44])
def test_a_wait_that_nothing_ends_gives_up_and_the_next_call_is_right(role, Hq, Nq, d):
    import exact_softmax_attention_fa_gb300 as fa
    lens = [1500, 300]
    p = filled(2, 1, d, 32, lens, BASE_SEED + role)
    qb, q = bf16(p.rng, 2, Hq, Nq, d)
    assert fa.fa_get_device_status_detail() == (0, 0, 0, 0)
    try:
        fa.fa_set_wait_limit_ns(2_000_000)
        fa.fa_debug_skip_arrival(role)
        call(p, qb, lens, None, True, scale_f32(d))
        code, where, block, _thread = fa.fa_get_device_status_detail()
    finally:
        fa.fa_debug_skip_arrival(0)
        fa.fa_set_wait_limit_ns(0)
    assert code == 6 and where in (41, 42, 43, 44) and block == 0
    o, lse = call(p, qb, lens, None, True, scale_f32(d))
    assert fa.fa_get_device_status_detail() == (0, 0, 0, 0)
    compare(p, q, lens, None, True, scale_f32(d), o, lse)


def test_a_cache_keeps_one_workspace_per_stream():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    gen = torch.Generator(device="cuda").manual_seed(BASE_SEED + 3)
    cache = fa.KV8Cache(2, 2, 64, 700)
    k = torch.randn(2, 2, 700, 64, generator=gen, device="cuda").bfloat16()
    cache.append(k, k)
    got = {}
    for Nq in (1, 40, 3, 300, 40, 1):
        q = torch.randn(2, 4, Nq, 64, generator=torch.Generator(device="cuda").manual_seed(Nq), device="cuda").bfloat16()
        o, lse = cache.attend(q)
        if Nq in got:
            assert torch.equal(o, got[Nq][0]) and torch.equal(lse, got[Nq][1])
        got[Nq] = o, lse
    assert len(cache._workspaces) == 1
    assert cache._workspaces.popitem()[1].numel() == max(fa.fa_fwd_kv8_workspace_size(2, 4, 2, n, 64) for n in got)
    assert fa.fa_get_device_status() == 0
