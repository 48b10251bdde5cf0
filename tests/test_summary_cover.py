"""A summary knows which blocks it holds: a choice over blocks that were never
summarised, or not since the cache grew, is refused instead of reading whatever
memory holds."""
from types import SimpleNamespace

import pytest
import torch

from test_blocks import query
from test_tree import kvq, make  # noqa: F401 (fixture)


def summary_of(kvq, cut, block=64):  # noqa: F811
    s = object.__new__(kvq.BlockSummary)
    s.cache, s.block = SimpleNamespace(cut=cut), block
    return s


def test_what_a_summary_covers(kvq):  # noqa: F811
    s = summary_of(kvq, 0)
    assert s.covers() and s.blocks == 0          # nothing to cover
    s.cache.cut = 200                            # 4 blocks, the last of 8 tokens
    assert not s.covers()
    s.filled(1)                                  # block 0 is still missing
    assert s.covers(1) and s.covers(3) and not s.covers()
    s.filled(0)
    assert s.covers()
    s.cache.cut = 232                            # the last block has more tokens now
    assert not s.covers() and not s.covers(3)
    s.filled(4)                                  # past the last: nothing
    assert not s.covers(3)
    s.filled(3)
    assert s.covers()
    s.cache.cut = 500                            # 8 blocks; 0 to 2 were whole
    s.filled(4)                                  # block 3 is left out
    assert not s.covers() and not s.covers(3) and s.covers(4)
    s.filled(3)
    assert s.covers(3) and not s.covers()        # (0 to 2: forgotten over the gap)
    s.filled()
    assert s.covers()
    s.cache.cut = 512
    s.filled(500 // 64)
    assert s.covers() and s.blocks == 8
    s.filled(8)                                  # nothing new: still covered
    s.filled(99)
    assert s.covers()
    s.cache.cut = 96                             # a shorter cache: its last block is another one
    assert not s.covers()
    s.filled(1)
    assert s.covers()


@pytest.mark.gpu
def test_choices_over_missing_summaries_are_refused(kvq):  # noqa: F811
    c = make(kvq, 1, 2, 704, 128, 64, reserve=(60, 160))
    s = kvq.BlockSummary(c, 64)
    q = query(1, 16, 1, 128)
    a = kvq.AttendBlocks(c, q, s, 3)
    for call in (a.run, s.values, lambda: kvq.attend_blocks(c, q, s, 3)):
        with pytest.raises(ValueError, match="cover"):
            call()
    s.update()
    want, sel = a.run().clone(), a.selected.clone()
    old = c.cut
    x = torch.randn((1, 2, 96, 128), device="cuda").bfloat16()
    kvq.append(c, x, x, 64)
    assert c.cut > old
    with pytest.raises(ValueError, match="cover"):
        a.run()
    assert torch.equal(a.out, want) and torch.equal(a.selected, sel)   # nothing ran
    a.run(select=False)                                                # the lists there: no summary
    s.update(first=old // 64)
    a.run()
    assert kvq.read_status(a.status) == 0 and int(a.selected.max()) < s.blocks
    # summaries of another origin
    t = kvq.BlockSummary(c, 64)
    t.codes.copy_(s.codes)
    t.scales.copy_(s.scales)
    t.filled()
    b = kvq.AttendBlocks(c, q, t, 3)
    assert torch.equal(b.run(), a.out) and torch.equal(b.selected, a.selected)


@pytest.mark.gpu
def test_no_summary_is_needed_to_take_every_block(kvq):  # noqa: F811
    c = make(kvq, 1, 2, 704, 128, 64, reserve=(60, 160))     # 10 blocks of 64
    s = kvq.BlockSummary(c, 64)                              # never updated
    q = query(1, 16, 1, 128)
    a = kvq.AttendBlocks(c, q, s, 10)
    out = a.run()
    assert kvq.read_status(a.status) == 0
    assert a.selected[0, 0, 0].tolist() == list(range(10))
    assert torch.equal(out, kvq.AttendBlocks(c, q, s.update(), 10).run())
    x = torch.randn((1, 2, 96, 128), device="cuda").bfloat16()
    kvq.append(c, x, x, 64)                                  # 12 blocks: now there is a choice
    with pytest.raises(ValueError, match="cover"):
        a.run()
