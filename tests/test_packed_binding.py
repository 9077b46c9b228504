"""What the binding of the packed operators refuses before it touches a device."""

import pytest

import exact_softmax_attention_fa_gb300 as fa

torch = pytest.importorskip("torch")


def plan_of(rows):
    """A PackedPlan as its constructor leaves it, without the device work."""
    plan = object.__new__(fa.PackedPlan)
    plan.rows, plan.causal, plan.B = rows, True, 1
    plan.buffer = torch.zeros(max(1, fa.fa_packed_plan_size(1, rows)), dtype=torch.uint8)
    return plan


@pytest.mark.parametrize("rows", [9, 11, 0])
def test_a_plan_of_other_rows_is_refused(rows):
    x, lse = torch.zeros(10, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 10)
    with pytest.raises(ValueError, match="rows"):
        fa.forward_packed(x, x, x, plan_of(rows))
    with pytest.raises(ValueError, match="rows"):
        fa.backward_packed(x, x, x, x, lse, x, plan_of(rows))
    with pytest.raises(ValueError, match="rows"):
        fa.backward_packed(x, x, x, x, lse, x, plan_of(rows), out=(x, x, x), workspace=torch.zeros(1, dtype=torch.uint8))
