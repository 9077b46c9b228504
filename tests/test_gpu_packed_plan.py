"""The plan of a packed batch as the calls take it: made for other rows, never made, dropped early."""

import pytest

from packed_util import Batch

pytestmark = pytest.mark.gpu

FA_ERR_INDEX = 8
SEED = 91000


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_plan_of_other_rows_or_none_leaves_everything_with_fill(d):
    """fill = 1 clears the rows of no sequence; a plan that is not of these rows says nothing about them."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([100, 30], 2, 2, d, SEED + d, tail=2)
    plan = fa.PackedPlan(b.d_cu, b.rows + 1)
    shape = (b.rows, 2, d)
    for p in (plan, torch.zeros_like(plan.buffer)):
        o, lse = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, b.rows), 7.0, device="cuda")
        fa.fa_fwd_packed(b.d_q, b.d_k, b.d_v, o, lse, p, True, 0.1, fill=True)
        assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 52)
        assert (o == 7).all() and (lse == 7).all()
        ws = torch.empty(fa.fa_bwd_packed_workspace_size(b.rows, 2, 2, d), dtype=torch.uint8, device="cuda")
        grads = [torch.full_like(o, 7.0) for _ in range(3)]
        fa.fa_bwd_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, *grads, p, True, 0.1, ws, fill=True)
        assert fa.fa_get_device_status_detail()[:2] == (FA_ERR_INDEX, 52)
        assert all((g == 7).all() for g in grads)


def test_forward_and_backward_refuse_a_plan_of_other_rows():
    import exact_softmax_attention_fa_gb300 as fa
    b = Batch([100, 30], 2, 2, 64, SEED, tail=2)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    o, lse = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan)
    fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan)
    for rows in (b.rows + 1, b.rows + 500):
        other = fa.PackedPlan(b.d_cu, rows)
        with pytest.raises(ValueError, match="rows"):
            fa.forward_packed(b.d_q, b.d_k, b.d_v, other)
        with pytest.raises(ValueError, match="rows"):
            fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, other)
    assert fa.fa_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_calls_behind_one_another_share_a_workspace(d):
    """Batches whose groups are split into different numbers of chunks take turns on one workspace: each call's kernels,
    which are resident before the ones they read from have ended, see this call's statistics, chunks and partial sums."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    Hq, Hkv = 8, 1
    batches = [Batch(lens, Hq, Hkv, d, SEED + 10 + i, tail=1100 - sum(lens), spread=1.0 + i)
               for i, lens in enumerate(([1000], [130] * 8, [5] * 100, [700, 300, 90]))]
    plans = [fa.PackedPlan(b.d_cu, b.rows) for b in batches]
    ws = torch.empty(fa.fa_bwd_packed_workspace_size(1100, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    alone = []
    for b, plan in zip(batches, plans):
        out = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan)
        ws.fill_(0xFF)  # NaN in the statistics and partial sums
        grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, *out, b.d_do, plan, workspace=ws)
        torch.cuda.synchronize()
        alone.append((out, grads))
    got = []
    for _ in range(10):
        for b, plan, (out, _) in zip(batches, plans, alone):
            got.append(fa.backward_packed(b.d_q, b.d_k, b.d_v, *out, b.d_do, plan, workspace=ws))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
    for i, grads in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(grads, alone[i % 4][1]))


def test_a_plan_dropped_while_another_stream_uses_it():
    """Made on one stream, used on another that is far behind, and dropped: nothing gets the plan's memory until then."""
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([300, 40, 129], 4, 2, 64, SEED + 30)
    want = fa.forward_packed(b.d_q, b.d_k, b.d_v, fa.PackedPlan(b.d_cu, b.rows))
    want_grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, *want, b.d_do, fa.PackedPlan(b.d_cu, b.rows))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = fa.PackedPlan(b.d_cu, b.rows)
    at, n = plan.buffer.data_ptr(), plan.buffer.numel()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    o, lse = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan, stream=side)
    grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, o, lse, b.d_do, plan, stream=side)
    del plan
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert not side.query()
    assert all(t.data_ptr() + n <= at or at + n <= t.data_ptr() for t in others)
    torch.cuda.synchronize()
    for x, y in zip((o, lse, *grads), (*want, *want_grads)):
        assert torch.equal(x, y)
    assert fa.fa_get_device_status() == 0


def test_a_plan_made_outside_serves_a_captured_step():
    import exact_softmax_attention_fa_gb300 as fa
    import torch
    b = Batch([300, 40, 129], 4, 2, 64, SEED + 31)
    plan = fa.PackedPlan(b.d_cu, b.rows)
    want = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan)
    want_grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, *want, b.d_do, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.forward_packed(b.d_q, b.d_k, b.d_v, plan)
        got_grads = fa.backward_packed(b.d_q, b.d_k, b.d_v, *got, b.d_do, plan)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((*got, *got_grads), (*want, *want_grads)):
            assert torch.equal(x, y)
            x.zero_()
    del graph, plan
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == 0
