"""A query row of NaN in the tensor-core chunk kernel: the row is NaN, the call
ends (its tile used to be redone without end), and the other rows are what they are
without it."""
import pytest
import torch


@pytest.mark.gpu
def test_nan_query_row_ends_and_stays_alone():
    from quantized_sparse_kv_gb300 import kvq
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((1, 2, 200, 128), generator=g, device="cuda").bfloat16()
    k = torch.randn((1, 2, 300, 128), generator=g, device="cuda").bfloat16()
    v = torch.randn((1, 2, 300, 128), generator=g, device="cuda").bfloat16()
    cache = kvq.pack(k, v, 300, "bf16")
    want, _, path = kvq.attend(cache, q, out_dtype="f32")
    assert path == "chunk_bf16"
    q[0, 1, 77] = torch.nan
    a = kvq.Attend(cache, q, out_dtype="f32")
    out = a.run()
    assert kvq.read_status(a.status) == 0
    assert bool(torch.isnan(out[0, 1, 77]).all())
    keep = torch.ones((1, 2, 200), dtype=torch.bool, device="cuda")
    keep[0, 1, 77] = False
    # a redone tile takes another reference: P is rounded to bf16 (2^-8) against it
    assert float((out[keep] - want[keep]).norm() / want[keep].norm()) <= 2.0 ** -8
