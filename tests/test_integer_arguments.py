"""Positions and parents are whole numbers: other types are refused, not cut."""
import pytest
import torch

from test_tree import kvq  # noqa: F401 (fixture)


@pytest.mark.parametrize("dt", [torch.float32, torch.float64, torch.bfloat16, torch.bool,
                                torch.complex64])
def test_positions_and_parents_of_other_types_are_refused(kvq, dt):  # noqa: F811
    plan = kvq.RopePlan(64, device="cpu")
    q = torch.zeros((1, 2, 3, 64))
    with pytest.raises(TypeError, match="positions"):
        kvq.Rope(plan, q, None, torch.zeros((1, 3)).to(dt))
    with pytest.raises(TypeError, match="parents"):
        kvq.AttendTree(None, q, q, q, torch.zeros((1, 3)).to(dt))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.int64, torch.int16, torch.uint8])
def test_positions_of_integer_types_are_taken(kvq, dt):  # noqa: F811
    plan = kvq.RopePlan(64)
    q = torch.randn((2, 2, 5, 64), device="cuda")
    pos = torch.arange(10, device="cuda", dtype=torch.int32).view(2, 5)
    want = kvq.rope(plan, q, None, pos)[0]
    assert torch.equal(kvq.rope(plan, q, None, pos.to(dt))[0], want)
