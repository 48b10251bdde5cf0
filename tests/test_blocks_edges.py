"""Attention over listed blocks where a row or a key holds NaN.

A row whose scores are NaN is NaN in every kernel, whatever the type of q and
however many partial results its keys give; rows beside it keep their bits, and
rows without keys stay zero.
"""
import pytest
import torch

from test_blocks import query
from test_tree import kvq, make  # noqa: F401 (fixture)

# b, hkv, n, window, block, blocks listed. Partials of a unit in the decode kernels (bf16 q, on
# 152 SMs): four; 17, merged by one warp in batches of 16; 65, merged by eight warps in batches
# of 8, so that the last partial, which holds the window's one key, has a batch to itself.
SLOTS = [(40, 2, 700, 64, 32, 5), (2, 2, 2500, 1, 32, 64), (1, 1, 9001, 1, 32, 256)]


def lists_of(b, hkv, nq, top, n_blocks):
    """The first `top` blocks for every list."""
    sel = torch.arange(top, dtype=torch.int32, device="cuda").clamp(max=n_blocks - 1)
    return sel.expand(b, hkv, nq, top).contiguous()


@pytest.mark.gpu
@pytest.mark.parametrize("case", SLOTS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_nan_query_row_is_nan_and_stays_alone(kvq, case, dt):  # noqa: F811
    b, hkv, n, window, block, top = case
    c = make(kvq, b, hkv, n, 128, window)
    q = query(b, 8 * hkv, 1, 128, dt)
    sel = lists_of(b, hkv, 1, top, -(-c.cut // block))
    a = kvq.AttendBlocks(c, q, None, top, out_dtype="f32", selected=sel, block=block)
    want = a.run(select=False).clone()
    assert a.path == ("blocks_decode" if dt == torch.bfloat16 else "blocks_rows")
    q[-1, 3, 0, 17] = torch.nan
    out = a.run(select=False)
    assert kvq.read_status(a.status) == 0
    assert bool(torch.isnan(out[-1, 3]).all())
    out[-1, 3], want[-1, 3] = 0.0, 0.0
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("case", SLOTS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_nan_key_reaches_every_row_that_attends_it(kvq, case, dt):  # noqa: F811
    b, hkv, n, window, block, top = case
    c = make(kvq, b, hkv, n, 128, window)
    q = query(b, 8 * hkv, 1, 128, dt)
    sel = lists_of(b, hkv, 1, top, -(-c.cut // block))
    a = kvq.AttendBlocks(c, q, None, top, out_dtype="f32", selected=sel, block=block)
    want = a.run(select=False).clone()
    c.k_window[0, hkv - 1, window - 1, 5] = torch.nan  # (with a window of one key: alone in its partial)
    out = a.run(select=False)
    assert kvq.read_status(a.status) == 0
    hit = slice(8 * (hkv - 1), 8 * hkv)
    assert bool(torch.isnan(out[0, hit]).all())
    out[0, hit], want[0, hit] = 0.0, 0.0
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,hkv", [(1, 1), (40, 2)])
def test_rows_without_keys_stay_zero_beside_nan_rows(kvq, dt, b, hkv):  # noqa: F811
    c = make(kvq, b, hkv, 13000, 128, 0) if b == 1 else make(kvq, b, hkv, 700, 128, 0)
    nq, top = 3, 406 if b == 1 else 5
    q = query(b, 8 * hkv, nq, 128, dt)
    sel = lists_of(b, hkv, nq, top, -(-c.cut // 32))
    sel[:, :, 1] = -1  # the second query token attends nothing
    a = kvq.AttendBlocks(c, q, None, top, out_dtype="f32", selected=sel, block=32)
    want = a.run(select=False).clone()
    assert not bool(want[:, :, 1].any())
    q[:, 0] = torch.nan  # the first head: NaN where it has keys
    out = a.run(select=False)
    assert kvq.read_status(a.status) == 0
    assert bool(torch.isnan(out[:, 0, 0]).all()) and bool(torch.isnan(out[:, 0, 2]).all())
    assert not bool(out[:, :, 1].any())
    assert torch.equal(out[:, 1:], want[:, 1:])


@pytest.mark.gpu
@pytest.mark.parametrize("b,n", [(1, 8193), (2, 2049), (40, 701)])
def test_a_nan_key_reaches_every_row_of_dense_decoding(kvq, b, n):  # noqa: F811
    c = make(kvq, b, 2, n, 128, 1)
    q = query(b, 16, 1, 128)
    a = kvq.Attend(c, q, out_dtype="f32")
    want = a.run().clone()
    assert a.path == "decode"
    c.k_window[0, 1, 0, 5] = torch.nan
    out = a.run()
    assert bool(torch.isnan(out[0, 8:]).all())
    out[0, 8:], want[0, 8:] = 0.0, 0.0
    assert torch.equal(out, want)
