"""kv_attend_pages on the tensor cores where magnitudes lie apart: tokens behind a row's
position. Against 64-bit attention over
the dequantized values; TOL_TENSOR as derived in test_pages.py (six roundings of 2^-11), which
holds wherever probabilities and scales keep their 11 bits.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kvq_oracle as O  # noqa: E402
from test_pages import TOL_TENSOR, attention64, kvq  # noqa: E402,F401
from test_pages_edges import one_request  # noqa: E402


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e3, 1e7, 1e9, 1e15, float("inf"), float("-inf"), float("nan")])
def test_tokens_behind_the_position_have_no_part(kvq, d, size):  # noqa: F811
    # rows that end inside an int4 group and inside a window tile, whose later tokens have
    # values of another size: what they see is as if the request ended there
    gen = torch.Generator(device="cuda").manual_seed(d)
    n, window = 640, 96
    for last in (489, 481, 510, 575, 600):
        k = torch.randn((n, 1, d), generator=gen, device="cuda")
        v = torch.randn((n, 1, d), generator=gen, device="cuda")
        v[last + 1:] = size
        k, v = k.bfloat16(), v.bfloat16()
        q = torch.randn((1, 8, d), generator=gen, device="cuda").bfloat16()
        with np.errstate(all="ignore"):
            cache, (kk, vv) = one_request(kvq, n, k, v, window, 1, d)
        call = kvq.AttendPages(cache, q, torch.zeros(1, dtype=torch.int32, device="cuda"),
                               torch.full((1,), last, dtype=torch.int32, device="cuda"),
                               out_dtype="f32")
        got = call.run().double().cpu().numpy()
        assert kvq.read_status(call.status) == 0 and call.path == "pages_tensor"
        want = attention64(q[0].double().cpu().numpy(), kk[:, :last + 1], vv[:, :last + 1])
        assert O.rel_l2(got[0], want) <= TOL_TENSOR, last
