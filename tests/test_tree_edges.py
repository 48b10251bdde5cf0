"""kv_attend_tree: hand-overs of short segments (tolerances as in test_tree.py)."""
import pytest
import torch

from test_tree import TOL_TENSOR, compare, inputs, kvq, make, plain, random_tree  # noqa: F401 (fixture)


@pytest.mark.gpu
@pytest.mark.parametrize("b,g,n,recent,t", [(250, 8, 100, 100, 5), (1000, 4, 60, 60, 1),
                                            (400, 8, 90, 0, 3), (170, 8, 100, 64, 16)])
def test_many_short_units_agree(kvq, b, g, n, recent, t):  # noqa: F811
    """Shared rows and one or two tiles a unit, several units a CTA: MMA warps without a step
    in a unit keep up with the others, run after run."""
    c = make(kvq, b, 2, n, 128, recent)
    q, k, v = inputs(b, 2 * g, 2, t, 128)
    par = random_tree(b, t, n + t)
    call = kvq.AttendTree(c, q, k, v, par, out_dtype="f32")
    first = call.run().clone()
    assert kvq.read_status(call.status) == 0 and call.path == "tree_tensor"
    compare(first, plain(c, kvq, q, k, v, par), par, TOL_TENSOR)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        differ += (call.run() != first).any()
    assert int(differ) == 0 and kvq.read_status(call.status) == 0
