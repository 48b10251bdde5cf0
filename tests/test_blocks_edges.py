"""Attention over listed blocks: rows and keys that hold NaN, and long lists.

A row whose scores are NaN is NaN in every kernel, whatever the type of q and
however many partial results its keys give; rows beside it keep their bits, and
rows without keys stay zero. Entries of a list past the number of blocks are not
looked at, wherever they fall among the four groups of an item. A key far above all
others leaves the others' probabilities their bits.
"""
import math

import pytest
import torch

from test_blocks import TOL_DECODE, TOL_F32, plain_attend, query, rel
from test_tree import dequant, kvq, make  # noqa: F401 (fixture)
from test_tree_edges import one_key_over_a_flat_tail

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


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block,blocks", [(64, 11), (64, 1), (32, 9), (32, 10), (32, 11), (128, 3)])
def test_entries_past_the_number_of_blocks_are_not_looked_at(kvq, dt, block, blocks):  # noqa: F811
    c = make(kvq, 1, 2, block * blocks, 128, 0)
    q = query(1, 16, 1, 128, dt)
    full = list(range(blocks))

    def run(row):
        sel = torch.tensor([[[row], [row]]], dtype=torch.int32, device="cuda")
        a = kvq.AttendBlocks(c, q, None, len(row), out_dtype="f32", selected=sel, block=block)
        out = a.run(select=False)
        return out.clone(), kvq.read_status(a.status)
    sel = torch.tensor([[[full], [full]]], dtype=torch.int32)
    want = plain_attend(c, kvq, q, sel, block)
    tol = TOL_DECODE if dt == torch.bfloat16 else TOL_F32
    for tail in ([99], [0], [blocks], [-2, 99, 3, 3], [-1, 0, 5]):
        out, st = run(full + tail)
        assert st == 0 and rel(out, want) <= tol, tail
    # the last entry looked at may still be bad
    out, st = run(full[:-1] + [blocks, 0, 0, 0])
    assert st == kvq.DEV_INDEX


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nats", [8.0, 12.0, 15.0, 16.0, 17.0, 18.0])
def test_a_key_far_above_a_flat_tail(kvq, dt, nats):  # noqa: F811
    """The decode kernels' P is fp16 against a reference 2^7 below a warp's maximum: at 18 nats
    the tail's P is 1.9e-6 in the warp that holds the first key, off by 2^-25 / 1.9e-6 = 1.6e-2
    of itself at most. That warp has a quarter of its unit's keys: 4e-3, and at 17 nats 1.4e-3;
    with the values' roundings (2^-11 twice, random) below 5e-3."""
    b, n = (128, 2048) if dt == torch.bfloat16 else (2, 2048)
    c, x, first = one_key_over_a_flat_tail(kvq, b, n, nats)
    q = torch.full((b, 16, 4, 128), x, device="cuda").to(dt)
    sel = lists_of(b, 2, 4, n // 64, n // 64)
    a = kvq.AttendBlocks(c, q, None, n // 64, sm_scale=math.log(2.0) / 8.0, out_dtype="f32",
                         selected=sel, block=64)
    out = a.run(select=False)
    assert kvq.read_status(a.status) == 0
    _, v = dequant(c, kvq)
    want = (v.sum(2) / (first + n - 1)).repeat_interleave(8, 1).unsqueeze(2).expand(out.shape)
    tol = TOL_DECODE if dt == torch.bfloat16 else TOL_F32
    assert float((out.double() - want).norm() / want.norm()) <= tol
