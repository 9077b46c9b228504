"""GPU parity of the attention over packed sequences (fa_packed_plan, fa_fwd_packed, fa_bwd_packed) against the 64-bit
reference of packed_util, whose bounds count the kernels' roundings element by element."""

import numpy as np
import pytest

from attn_inputs import BASE_SEED
from gpu_util import scale_f32, to_host64
from packed_util import Batch, backward_ref, forward_ref, starts, within

pytestmark = pytest.mark.gpu

FA_ERR_TIMEOUT, FA_ERR_INDEX = 6, 8


def run(b, causal, scale, plan=None):
    import exact_softmax_attention_fa_gb300 as fa
    plan = plan or fa.PackedPlan(b.d_cu, b.rows, causal)
    o, lse = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, scale=scale)
    grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan, scale=scale)
    assert fa.fa_get_device_status_detail() == (0, 0, 0, 0)
    return o, lse, grads


def check(b, causal):
    scale = scale_f32(b.d)
    o, lse, grads = run(b, causal, scale)
    held = b.held()
    ho, hl = to_host64(o), lse.cpu().numpy().astype(np.float64)
    o_ref, l_ref, bo, bl = forward_ref(b, causal, scale)
    assert within(ho, o_ref, bo, held) <= 1.0
    assert within(hl.T, l_ref.T, bl.T, held) <= 1.0
    ref, bound = backward_ref(b, ho, hl, causal, scale)
    for name, g, r, e in zip(("dq", "dk", "dv"), grads, ref, bound):
        assert within(to_host64(g), r, e, held) <= 1.0, name
    for t in (ho, *(to_host64(g) for g in grads)):
        assert (t[~held] == 0).all()
    assert (hl[:, ~held] == 0).all()


LENS = [[1], [1, 2, 15, 16, 17], [127, 128, 129], [0, 40, 0, 0, 300, 3, 0], [255, 256, 257, 31], [64] * 9, [640, 385]]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_parity(lens, causal, d):
    check(Batch(lens, 4, 2, d, BASE_SEED + sum(lens)), causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (8, 1), (6, 2), (16, 8)])
def test_heads(Hq, Hkv, causal, d):
    check(Batch([130, 1, 77, 259], Hq, Hkv, d, BASE_SEED + Hq, lead=5, tail=19), causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_many_sequences(d, causal):
    # more items than SMs, in every amount of work, some sequences empty
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 200, 150)] + [700, 1025]
    check(Batch(lens, 2, 1, d, BASE_SEED + 900, tail=3), causal)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 1), (64, 4, 4), (256, 2, 1)])
def test_long_sequence_beside_short_ones(d, Hq, Hkv):
    check(Batch([3, 2600, 50, 1], Hq, Hkv, d, BASE_SEED + 950), True)


def test_split_groups():
    # one short sequence of few K/V heads: a group's heads go to several SMs, whose sums are joined
    check(Batch([1500], 8, 1, 128, BASE_SEED + 960, lead=1, tail=1), True)
    check(Batch([700, 20], 6, 1, 64, BASE_SEED + 961), False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1)])
def test_around_the_short_kernels_limit(Hq, Hkv, causal, d):
    check(Batch([63, 65, 64, 66, 1, 62], Hq, Hkv, d, BASE_SEED + 970), causal)


def test_layouts():
    """Heads outside, tokens outside, and a packed projection: the same bits."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([200, 57, 129], 4, 2, 128, BASE_SEED + 10)
    o, lse, grads = run(b, True, 0.1)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    heads = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (b.d_q, b.d_k, b.d_v, b.d_do)]
    out = torch.empty(4, b.rows, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    l2 = torch.empty_like(lse)
    fa.fa_fwd_packed(*heads[:3], out, l2, plan, True, 0.1)
    packed = torch.empty_like(b.qkv)
    views = packed[:, :4], packed[:, 4:6], packed[:, 6:]
    fa.backward_packed(*heads[:3], out, l2, heads[3], plan, scale=0.1, out=views)
    assert torch.equal(out, o) and torch.equal(l2, lse)
    for a, c in zip(views, grads):
        assert torch.equal(a, c)


def test_a_single_sequence_is_the_dense_call():
    """The same bits, but for dQ and dK: their dS takes weights in fp32 instead of bf16."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([515], 3, 3, 128, BASE_SEED + 11)
    o, lse, (dq, dk, dv) = run(b, True, 0.1)
    dense = [t.transpose(0, 1)[None].contiguous() for t in (b.d_q, b.d_k, b.d_v, b.d_do)]
    o2, l2 = fa.forward(*dense[:3], causal=True, scale=0.1)
    assert torch.equal(o2[0].transpose(0, 1), o) and torch.equal(l2[0], lse)
    dense_grads = fa.backward(*dense[:3], o2, l2, dense[3], causal=True, scale=0.1)
    assert torch.equal(dense_grads[2][0].transpose(0, 1), dv)
    ref, _ = backward_ref(b, to_host64(o), lse.cpu().numpy().astype(np.float64), True, float(np.float32(0.1)))
    for a, g, r in zip(dense_grads, (dq, dk), ref):
        assert np.linalg.norm(to_host64(g) - r) < np.linalg.norm(to_host64(a[0].transpose(0, 1)) - r)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_other_sequences_have_no_effect(d, causal):
    """NaN and infinities all through the neighbours, before and behind, leave every bit as it was."""
    import torch
    b = Batch([90, 141, 5, 200], 4, 2, d, BASE_SEED + 12, lead=7, tail=9)
    o, lse, grads = run(b, causal, 0.1)
    for keep in (1, 2):
        r = slice(int(b.cu[keep]), int(b.cu[keep + 1]))
        for t in (b.qkv, b.d_do):
            was = t[r].clone()
            t[..., ::2] = float("nan")
            t[..., 1::2] = float("-inf")
            t[r] = was
        o2, l2, g2 = run(b, causal, 0.1)
        assert torch.equal(o2[r], o[r]) and torch.equal(l2[:, r], lse[:, r])
        for x, y in zip(g2, grads):
            assert torch.equal(x[r], y[r])
        b = Batch([90, 141, 5, 200], 4, 2, d, BASE_SEED + 12, lead=7, tail=9)


def test_rows_of_no_sequence_are_left():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([130, 0, 61], 2, 1, 64, BASE_SEED + 13, lead=70, tail=200)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    o = torch.full((b.rows, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, b.rows), 7.0, device="cuda")
    fa.fa_fwd_packed(b.d_q, b.d_k, b.d_v, o, lse, plan, True, 0.1)
    grad = torch.full_like(b.qkv, 7.0)
    ws = torch.empty(fa.fa_bwd_packed_workspace_size(b.rows, 2, 1, 64), dtype=torch.uint8, device="cuda")
    fa.fa_bwd_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, grad[:, :2], grad[:, 2:3], grad[:, 3:], plan, True, 0.1, ws)
    assert fa.fa_get_device_status() == 0
    out = torch.tensor(~b.held(), device="cuda")
    for t in (o, lse.T, grad):
        assert (t[out] == 7).all()
        assert not t[~out].isnan().any()
    # the smallest workspace rules out split groups, nothing else
    least = torch.empty(256 + 2 * (-(-4 * b.rows * 2 // 256) * 256), dtype=torch.uint8, device="cuda")
    again = torch.full_like(b.qkv, 7.0)
    fa.fa_bwd_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, again[:, :2], again[:, 2:3], again[:, 3:], plan, True, 0.1,
                     least)
    # (a sum over the heads in one piece instead of two: other roundings, the same bounds)
    assert torch.equal(grad[:, :2], again[:, :2]) and (again[out] == 7).all()
    ref, bound = backward_ref(b, to_host64(o), lse.cpu().numpy().astype(np.float64), True, float(np.float32(0.1)))
    for got in (grad, again):
        for t, r, e in zip((got[:, :2], got[:, 2:3], got[:, 3:]), ref, bound):
            assert within(to_host64(t), r, e, b.held()) <= 1.0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_results_do_not_depend_on_the_plans_order(d):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([300, 17, 1, 128, 555, 64], 8, 2, d, BASE_SEED + 14)
    first = run(b, True, 0.1)
    for causal in (True, False, True):
        plan = fa.PackedPlan(b.d_cu, b.rows, causal)
        o, lse = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, True, 0.1)
        grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan, True, 0.1)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
        for x, y in zip(grads, first[2]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [-1, 10, 20, 30], [0, 10, 20, 301], [5, 4, 4, 4], [0, 2**31 - 1, 5, 9]])
def test_lengths_out_of_range(cu):
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([100, 100, 100], 2, 2, 64, BASE_SEED + 15)
    plan = fa.PackedPlan(torch.tensor(cu, dtype=torch.int32, device="cuda"), b.rows)
    assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 51)
    o, lse = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, scale=0.1)
    assert (o == 0).all() and (lse == 0).all()  # a plan without sequences
    grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan, scale=0.1)
    assert all((g == 0).all() for g in grads)
    assert fa.fa_get_device_status() == 0
    plan.update(b.d_cu)
    o, _ = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, scale=0.1)
    assert torch.equal(o, run(b, True, 0.1)[0])


def test_a_plan_of_other_rows_or_none_is_refused():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([100, 30], 2, 2, 64, BASE_SEED + 16, tail=2)
    plan = fa.PackedPlan(b.d_cu, b.rows + 1)
    o = torch.full((b.rows, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, b.rows), 7.0, device="cuda")
    for p in (plan, torch.zeros_like(plan.buffer)):
        fa.fa_fwd_packed(b.d_q, b.d_k, b.d_v, o, lse, p, True, 0.1)
        assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 52)
        assert (o == 7).all() and (lse == 7).all()
        ws = torch.empty(fa.fa_bwd_packed_workspace_size(b.rows, 2, 2, 64), dtype=torch.uint8, device="cuda")
        grads = [torch.full_like(o, 7.0) for _ in range(3)]
        fa.fa_bwd_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, *grads, p, True, 0.1, ws)
        assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 52)
        assert all((g == 7).all() for g in grads)


def test_empty_calls():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    for cu in ([0], [0, 0, 0]):
        plan = fa.PackedPlan(torch.tensor(cu, dtype=torch.int32, device="cuda"), 0)
        o, lse = fa.forward_packed(none, none, none, plan)
        assert o.shape == none.shape and lse.shape == (2, 0)
        fa.backward_packed(none, none, none, o, lse, none, plan)
    x = torch.randn(9, 2, 64, device="cuda").bfloat16()
    plan = fa.PackedPlan(torch.tensor([4, 4, 4], dtype=torch.int32, device="cuda"), 9)
    o, lse = fa.forward_packed(x, x, x, plan)
    assert (o == 0).all() and (lse == 0).all()
    assert all((g == 0).all() for g in fa.backward_packed(x, x, x, o, lse, x, plan))
    assert fa.fa_get_device_status() == 0


def test_captured_step_replays_with_other_lengths():
    """Plan, forward and backward in one graph; another batch's lengths and values go into the same memory."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    batches = [Batch(lens, 4, 2, 128, BASE_SEED + 20 + i, tail=t) for i, (lens, t) in
               enumerate((([100, 300, 50, 0], 0), ([449, 1, 0, 0], 0), ([7, 9, 11, 13], 410)))]
    b = batches[0]
    plan = fa.PackedPlan(b.d_cu, b.rows)
    run(b, True, 0.1, plan)
    qkv, do, cu = b.qkv.clone(), b.d_do.clone(), b.d_cu.clone()
    views = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.update(cu)
        o, lse = fa.forward_packed(*views, plan, scale=0.1)
        grads = fa.backward_packed(*views, o, lse, do, plan, scale=0.1)
    for x in batches[1:] + batches[:1]:
        qkv.copy_(x.qkv), do.copy_(x.d_do), cu.copy_(x.d_cu)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, lse, *grads)]
        want = run(x, True, 0.1)
        for a, c in zip(got, (want[0], want[1], *want[2])):
            assert torch.equal(a, c)


def test_graphs_of_two_batches_share_a_workspace():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    bs = [Batch(lens, 8, 2, 128, BASE_SEED + 25 + i) for i, lens in enumerate(([700, 40, 260], [10, 600, 64, 65, 261]))]
    want = [run(b, True, 0.1) for b in bs]
    assert bs[0].rows == bs[1].rows
    ws = torch.empty(fa.fa_bwd_packed_workspace_size(1000, 8, 2, 128), dtype=torch.uint8, device="cuda")
    made = []
    for b in bs:
        plan = fa.PackedPlan(b.d_cu, b.rows)
        o, lse, grad = torch.empty_like(b.d_do), torch.empty(8, b.rows, device="cuda"), torch.empty_like(b.qkv)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.fa_fwd_packed(b.d_q, b.d_k, b.d_v, o, lse, plan, True, 0.1)
            fa.fa_bwd_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, grad[:, :8], grad[:, 8:10], grad[:, 10:], plan, True,
                             0.1, ws)
        made.append((graph, plan, o, lse, grad))
    for _ in range(3):
        for graph, _, o, lse, grad in made:
            for t in (o, lse, grad):
                t.fill_(7.0)
            graph.replay()
        torch.cuda.synchronize()
        for (_, _, o, lse, grad), w in zip(made, want):
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
            for x, y in zip((grad[:, :8], grad[:, 8:10], grad[:, 10:]), w[2]):
                assert torch.equal(x, y)


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 1, 128), (8, 8, 64), (4, 1, 256)])
def test_work_queued_behind_sees_final_results(Hq, Hkv, d):
    """The kernels of a call overlap each other; copies queued right behind it are of what all of them have written."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([1200, 30, 64, 5, 500] + [20] * 100, Hq, Hkv, d, BASE_SEED + 35)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    o, lse = torch.empty_like(b.d_do), torch.empty(Hq, b.rows, device="cuda")
    grad = torch.empty_like(b.qkv)
    ws = torch.empty(fa.fa_bwd_packed_workspace_size(b.rows, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    copies = []
    for _ in range(12):
        for t in (o, lse, grad):
            t.fill_(7.0)
        fa.fa_fwd_packed(b.d_q, b.d_k, b.d_v, o, lse, plan, True, 0.1)
        kept = [o.clone(), lse.clone()]
        fa.fa_bwd_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, grad[:, :Hq], grad[:, Hq:Hq + Hkv], grad[:, Hq + Hkv:], plan,
                         True, 0.1, ws)
        copies.append(kept + [grad.clone()])
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    for c in copies:
        for x, y in zip(c, (o, lse, grad)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_further_apart_than_32_bits(d):
    """Every tensor a view of one whose rows lie 2^24 elements apart: the last rows are 2^31 elements behind the
    first and more. The same bits as from tensors of their own."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    Hq, Hkv = 4, 2
    b = Batch([140, 20, 1], Hq, Hkv, d, BASE_SEED + 36)
    want = run(b, True, 0.1)
    wide = torch.empty(b.rows << 24, dtype=torch.bfloat16, device="cuda")
    place = [0]

    def view(heads):
        t = wide.as_strided((b.rows, heads, d), (1 << 24, d, 1), place[0])
        place[0] += heads * d
        return t

    q, k, v, do, o, dq, dk, dv = (view(h) for h in (Hq, Hkv, Hkv, Hq, Hq, Hq, Hkv, Hkv))
    for t, x in ((q, b.d_q), (k, b.d_k), (v, b.d_v), (do, b.d_do)):
        t.copy_(x)
    plan, lse = fa.PackedPlan(b.d_cu, b.rows), torch.empty(Hq, b.rows, device="cuda")
    ws = torch.empty(fa.fa_bwd_packed_workspace_size(b.rows, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    fa.fa_fwd_packed(q, k, v, o, lse, plan, True, 0.1)
    fa.fa_bwd_packed(q, k, v, o, lse, do, dq, dk, dv, plan, True, 0.1, ws)
    assert fa.fa_get_device_status() == 0
    for x, y in zip((o, lse, dq, dk, dv), (want[0], want[1], *want[2])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_every_sm_busy_for_long(causal, d):
    """Many items of many tiles on every SM, where the warps of a kernel drift apart as far as they can: no wait gives
    up, every run has the same bits, and O, L and dV those of the dense call."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    lens, H = [2900, 4096, 1999, 3500, 2333, 3201], 12
    g = torch.Generator(device="cuda").manual_seed(BASE_SEED + 980 + d)
    x = torch.randn(sum(lens), 4 * H, d, generator=g, device="cuda").bfloat16()
    q, k, v, do = x.split(H, 1)
    cu = torch.tensor(starts(lens), device="cuda")
    plan = fa.PackedPlan(cu, sum(lens), causal)
    first = None
    for _ in range(3):
        o, lse = fa.forward_packed(q, k, v, plan)
        got = (o, lse, *fa.backward_packed(q, k, v, o, lse, do, plan))
        assert fa.fa_get_device_status_detail() == (0, 0, 0, 0)
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b)
    for r in (slice(0, 2900), slice(8995, 12495)):
        one = [t[r].transpose(0, 1)[None].contiguous() for t in (q, k, v, do)]
        o2, l2 = fa.forward(*one[:3], causal=causal)
        dv2 = fa.backward(*one[:3], o2, l2, one[3], causal=causal)[2]
        assert torch.equal(o2[0].transpose(0, 1), first[0][r]) and torch.equal(l2[0], first[1][:, r])
        assert torch.equal(dv2[0].transpose(0, 1), first[4][r])


def test_two_streams_share_a_plan():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    bs = [Batch([400, 33, 129, 600], 4, 2, 64, BASE_SEED + 30 + i) for i in range(2)]
    plan = fa.PackedPlan(bs[0].d_cu, bs[0].rows)
    want = [run(b, True, 0.1, plan) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (b, s) in enumerate(zip(bs, streams)):
            o, lse = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, scale=0.1, stream=s)
            got[i].append((o, lse, *fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan, scale=0.1, stream=s)))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    for i, w in enumerate(want):
        for g in got[i]:
            for x, y in zip(g, (w[0], w[1], *w[2])):
                assert torch.equal(x, y)


def test_scores_out_of_the_ordinary():
    """Rows whose scores are all far below zero, all equal, or spread over hundreds: one key takes all."""
    b = Batch([200, 129], 2, 1, 64, BASE_SEED + 40, spread=12.0)
    check(b, True)
    b = Batch([200, 129], 2, 1, 64, BASE_SEED + 41)
    b.qkv[:, :2] = 0  # equal scores: the mean of the values
    b.x[:, :2] = 0
    check(b, False)


def test_binding_refuses():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([100], 4, 2, 64, BASE_SEED + 50)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    o, lse, _ = run(b, True, 0.1, plan)
    call = lambda **kw: fa.fa_fwd_packed(*(kw.get(n, t) for n, t in (
        ("q", b.d_q), ("k", b.d_k), ("v", b.d_v), ("o", o), ("lse", lse), ("plan", plan))), True, 0.1)
    call()
    with pytest.raises(TypeError):
        call(q=b.d_q.float())
    for bad in (dict(k=b.d_k[:50]), dict(q=b.d_q[:, :3], o=o[:, :3]), dict(v=b.d_v.transpose(1, 2)), dict(o=o[:, :, :32]),
                dict(lse=lse.T), dict(lse=lse.double()), dict(q=b.d_q[0]), dict(o=o.cpu()), dict(plan=plan.buffer[::2])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(fa.FAError):  # a row's values not at a 16-byte boundary
        call(q=torch.empty(100 * 4 * 72 + 8, dtype=torch.bfloat16, device="cuda")[4:28804].view(100, 4, 72)[:, :, :64])
    with pytest.raises(fa.FAError):  # heads that overlap in the output
        call(o=torch.empty(103 * 64, dtype=torch.bfloat16, device="cuda").as_strided((100, 4, 64), (64, 64, 1)))
    with pytest.raises(fa.FAError):  # rows that are one
        call(k=b.d_k[:1].expand(100, 2, 64))
    with pytest.raises(ValueError):
        fa.PackedPlan(b.d_cu.long(), b.rows)
    with pytest.raises(ValueError):
        fa.fa_packed_plan(b.d_cu.cpu(), b.rows, True, plan.buffer)
    with pytest.raises(fa.FAError):
        fa.fa_packed_plan(b.d_cu, b.rows, True, plan.buffer[:256])
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("d,role", [(128, 1), (128, 2), (128, 3), (64, 11), (128, 12), (64, 13), (256, 11), (256, 12),
                                    (256, 13)])
def test_waits_give_up_and_the_next_call_is_right(cuda_lib, d, role):
    import exact_softmax_attention_fa_gb300 as fa
    b = Batch([300, 17, 513], 4, 2, d, BASE_SEED + 60)
    o, lse, _ = run(b, True, 0.1)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    try:
        fa.fa_set_wait_limit_ns(2_000_000)
        fa.fa_debug_skip_arrival(role)
        if role < 10:
            fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, scale=0.1)
        else:
            fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan, scale=0.1)
        code, where, block, _ = fa.fa_get_device_status_detail()
    finally:
        fa.fa_debug_skip_arrival(0)
        fa.fa_set_wait_limit_ns(0)
    assert code == FA_ERR_TIMEOUT and block == 0 and (where < 10) == (role < 10)
    check(b, True)
