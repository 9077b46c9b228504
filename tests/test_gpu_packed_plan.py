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
