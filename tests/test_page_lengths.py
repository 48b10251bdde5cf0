"""Which lengths a request of the paged cache may have, on the CPU.

paged.cuh is compiled as a host program: PagedDims::holds against the rule in 64 bits (the
pages of cut(L) are at most max_pages) for lengths at both ends of 32 bits and around
every limit, whatever an array of lengths contains. On the GPU: such lengths are flagged
and nothing is read or written for them.
"""
import ctypes
import os
import shutil
import subprocess
import textwrap

import pytest

torch = pytest.importorskip("torch")

from test_pages import kvq, poison  # noqa: E402,F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_sparse_kv_gb300", "csrc")

_PROGRAM = textwrap.dedent(r"""
    #include <cstdio>
    #include <initializer_list>
    #include "paged.cuh"
    int main() {
      long checked = 0, bad = 0;
      for (int log2 : {5, 6, 7})
        for (int window : {0, 1, 31, 33, 128, 65536})
          for (long pages : {1L, 6L, 1000L, ((1L << 31) - 1 - window - 64) >> log2}) {
            kvq::PagedDims d = {};
            d.page_log2 = log2;
            d.window = window;
            d.max_pages = static_cast<int>(pages);
            const long top = (pages << log2) + window;
            for (long base : {0L, top, 1L << 30, (1L << 31) - 1})
              for (long len = base - 300; len <= base + 300; ++len) {
                if (len < -(1L << 31) || len > (1L << 31) - 1) continue;
                const long cut = len >= window ? (len - window) / 32 * 32 : 0;
                const bool want = len >= 0 && (cut + (1L << log2) - 1) >> log2 <= pages;
                ++checked;
                bad += d.holds(static_cast<int>(len)) != want;
              }
            bad += d.holds(-2147483647 - 1);
          }
      std::printf("%ld %ld\n", checked, bad);
      return 0;
    }
""")


def test_lengths_that_a_table_holds(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "holds_check.cu"
    src.write_text(_PROGRAM)
    exe = tmp_path / "holds_check"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    checked, bad = map(int, out)
    assert checked > 100000 and bad == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(128, "bf16"), (32, "f32")])
@pytest.mark.parametrize("page", [32, 64, 128])
def test_lengths_that_no_table_holds_are_flagged(kvq, page, d, wdt):  # noqa: F811
    state = kvq.PageState(3, 6, page, 6, 0)
    cache = kvq.PagedCache(state, 1, d, wdt)
    poison(cache)
    x = torch.randn((40, 1, d), device="cuda")
    kvq.append_pages(cache, kvq.page_tables(state, torch.tensor([40, 0, 0], device="cuda"), 40), x, x)
    assert int(state.n_free[0]) == 6 - state.pages(40)
    for length in ((1 << 31) - 1, (1 << 31) - 33, (1 << 31) - 128, -1, -(1 << 31), 6 * page + 32):
        state.lengths[1] = length
        for n_new in (0, 1, -1):
            plan = kvq.page_tables(state, torch.tensor([0, n_new, 0], device="cuda"), 1)
            assert kvq.read_status(plan.status) == kvq.DEV_INDEX
            assert state.lengths.tolist() == [40, length, 0]
            assert plan.row_slot.tolist() == [-1]
            assert int(state.n_free[0]) == 6 - state.pages(40)
        q = torch.randn((2, 2, d), device="cuda")
        slot = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
        for pos in (None, torch.tensor([0, 3], dtype=torch.int32, device="cuda")):
            out = torch.full(q.shape, 3.0, device="cuda")
            call = kvq.AttendPages(cache, q, slot, pos, out=out)
            call.run()
            assert kvq.read_status(call.status) == kvq.DEV_INDEX
            assert bool((out[0] == 3.0).all()) and bool((out[1] != 3.0).all())
        vals = kvq.PageValues(cache, slot, torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
        vals.run()
        assert kvq.read_status(vals.status) == kvq.DEV_INDEX
        assert bool((vals.k[0] == 0).all()) and bool((vals.k[1] != 0).any())


def test_sizes_that_64_bits_do_not_hold_are_refused(kvq):  # noqa: F811
    lib = kvq.load_library()
    sizes = (ctypes.c_size_t * 6)()
    state = kvq.KvqPageState(8192, 1 << 28, 128, 1000, 65536)
    # the largest that is taken, then one whose pool would have 2^64 bytes and more
    assert lib.kvq_paged_sizes(ctypes.byref(kvq.KvqPagedCache(state, 65535, 256, 0)), sizes) == 0
    assert sizes[4] == (1 << 28) * 65535 * 4 * 40 * 256
    assert sizes[5] == 8192 * 65535 * 2049 * 2 * 32 * 256 * 4
    for heads in (65536, 1 << 30, (1 << 31) - 1):
        assert lib.kvq_paged_sizes(ctypes.byref(kvq.KvqPagedCache(state, heads, 256, 0)), sizes) == 1


def test_more_values_than_a_grid_has_blocks_are_refused(kvq):  # noqa: F811
    lib, addr = kvq.load_library(), 1 << 20
    state = kvq.KvqPageState(4, 10, 64, 5, 128, addr, addr, addr, addr)
    cache = kvq.KvqPagedCache(state, 65, 128, 1, addr, addr)
    assert lib.kv_page_values(ctypes.byref(cache), addr, addr, 1 << 28, addr, addr, 1, None,
                              None) == 3
