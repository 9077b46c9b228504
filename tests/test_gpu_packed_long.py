"""Packed sequences of more tiles than the plan has bins of work: the lists themselves, and sampled rows of both passes."""

import numpy as np
import pytest

from gpu_util import scale_f32, to_host64
from packed_util import H16, TINY, starts

pytestmark = pytest.mark.gpu

SEED, BINS, SHORT = 93000, 2048, 64


def lists(plan):
    """The head of a plan and its two lists of {first row, length, index, 0}."""
    raw = plan.buffer.cpu().numpy().tobytes()
    head = np.frombuffer(raw, np.int32, 9)
    n_tiles, n_pairs, pairs_at = int(head[2]), int(head[3]), int(head[5])
    entries = np.frombuffer(raw, np.int32, offset=256)[: 4 * (pairs_at + n_pairs)].reshape(-1, 4)
    products = np.frombuffer(raw, np.uint64, 2, offset=40)
    return head, products, entries[:n_tiles], entries[pairs_at:pairs_at + n_pairs]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[BINS * 128 - 129], [BINS * 128 - 128], [BINS * 128], [5, 300000, 0, 64, 65, 1000, 262017, 1],
                                  [4 * BINS * 128 + 7, 70], [63] * 1500 + [1200] * 40], ids=lambda x: str(x[:3]))
def test_every_tile_once_and_the_most_work_first(lens, causal):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    cu = starts(lens, 3)
    plan = fa.PackedPlan(torch.tensor(cu, device="cuda"), int(cu[-1]) + 4, causal)
    head, products, tiles, pairs = lists(plan)
    T = [-(-n // 128) for n in lens]
    assert head[6] == max(T) and head[7] == 3 and head[8] == cu[-1]
    assert head[4] == sum(0 < n <= SHORT for n in lens)
    assert list(products) == [sum(t * (t + 1) // 2 for t in T), sum(t * t for t in T)]
    shift = 0
    while -(-max(T) >> shift) >= BINS:
        shift += 1
    for got, per in ((tiles, 1), (pairs, 2)):
        want = {(int(c), n, i) for c, n, t in zip(cu, lens, T) for i in range(-(-t // per))}
        assert len(got) == len(want) and {tuple(int(y) for y in x[:3]) for x in got} == want
        n, t, i = got[:, 1], -(-got[:, 1] // 128), got[:, 2]
        seen = np.where(n <= SHORT, 0, np.minimum(per * (i + 1), t) if causal else t)
        work = -(-seen >> shift)  # sequences longer than the bins share them
        assert (np.diff(work) <= 0).all()
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1)])
def test_sampled_rows_of_a_long_sequence(Hq, Hkv):
    """As packed_util, and n / 16 additions of 16 products each to an fp32 sum, 2^-23 of the terms so far each."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    d, n, lead = 64, BINS * 128 + 300, 40
    g = torch.Generator(device="cuda").manual_seed(SEED + Hq)
    x = torch.randn(lead + n + 9, Hq + 2 * Hkv, d, device="cuda", generator=g).bfloat16()
    do = torch.randn(lead + n + 9, Hq, d, device="cuda", generator=g).bfloat16()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    plan = fa.PackedPlan(torch.tensor([0, lead, lead + n], dtype=torch.int32, device="cuda"), len(x))
    scale = scale_f32(d)
    o, lse = fa.forward_packed(q, k, v, plan, scale=scale)
    dq, dk, dv = fa.backward_packed(q, k, v, o, lse, do, plan, scale=scale)
    assert fa.fa_get_device_status_detail() == (0, 0, 0, 0)
    s = slice(lead, lead + n)
    hq, hk, hv, hdo, ho = (to_host64(t[s]) for t in (q, k, v, do, o))
    hl = lse[:, s].double().cpu().numpy()
    got_q, got_k, got_v = (to_host64(t[s]) for t in (dq, dk, dv))
    rows = np.unique(np.concatenate([[0, 1, 127, 128, n - 301, n - 2, n - 1],
                                     np.random.default_rng(SEED).integers(0, n, 12)]))
    long = n / 16 * 2.0 ** -23
    D = (hdo * ho).sum(-1)
    for h in range(Hq):
        for i in rows:
            seen = slice(0, i + 1)
            sc, mag = scale * (hk[seen, 0] @ hq[i, h]), scale * (np.abs(hk[seen, 0]) @ np.abs(hq[i, h]))
            m = sc.max()
            p = np.exp(sc - m)
            l = p.sum()
            p /= l
            off = d * 2.0 ** -23 * mag.max()
            ref = p @ hv[seen, 0]
            bound = H16 * np.abs(ref) + (H16 + 2 * off + 2.0 ** -18 + 2 * long) * (p @ np.abs(hv[seen, 0]))
            assert (np.abs(ho[i, h] - ref) <= bound).all(), i
            L = m + np.log(l)
            assert abs(hl[h, i] - L) <= off + long + 2.0 ** -18 * (1 + abs(L)), i
            p = np.exp(sc - hl[h, i])
            dp = hv[seen, 0] @ hdo[i, h]
            ds = p * (dp - D[i, h])
            rel = off + 2.0 ** -23 * abs(hl[h, i]) + 2.0 ** -18
            e = d * 2.0 ** -23 * (np.abs(hv[seen, 0]) @ np.abs(hdo[i, h]) + (np.abs(hdo[i, h]) * np.abs(ho[i, h])).sum())
            ds_off = (H16 + rel + long) * np.abs(ds) + 1.01 * p * e + TINY * (1 + np.abs(dp - D[i, h]))
            ref = scale * (ds @ hk[seen, 0])
            assert (np.abs(got_q[i, h] - ref) <= H16 * np.abs(ref) + 1.01 * scale * (ds_off @ np.abs(hk[seen, 0]))).all(), i
    for j in rows:
        ref_k, ref_v, bound_k, bound_v = (np.zeros(d) for _ in range(4))
        for h in range(Hq):
            seen = slice(j, n)
            sc, mag = scale * (hq[seen, h] @ hk[j, 0]), scale * (np.abs(hq[seen, h]) @ np.abs(hk[j, 0]))
            p = np.exp(sc - hl[h, seen])
            dp = hdo[seen, h] @ hv[j, 0]
            ds = p * (dp - D[seen, h])
            rel = d * 2.0 ** -23 * mag + 2.0 ** -23 * np.abs(hl[h, seen]) + 2.0 ** -18 + Hq * long
            e = d * 2.0 ** -23 * (np.abs(hdo[seen, h]) @ np.abs(hv[j, 0])
                                  + (np.abs(hdo[seen, h]) * np.abs(ho[seen, h])).sum(-1))
            ds_off = (H16 + rel) * np.abs(ds) + 1.01 * p * e + TINY * (1 + np.abs(dp - D[seen, h]))
            ref_k += scale * (ds @ hq[seen, h])
            bound_k += 1.01 * scale * (ds_off @ np.abs(hq[seen, h]))
            ref_v += p @ hdo[seen, h]
            bound_v += 1.01 * (((H16 + rel) * p + TINY) @ np.abs(hdo[seen, h]))
        assert (np.abs(got_k[j, 0] - ref_k) <= bound_k + H16 * np.abs(ref_k)).all(), j
        assert (np.abs(got_v[j, 0] - ref_v) <= bound_v + H16 * np.abs(ref_v)).all(), j
