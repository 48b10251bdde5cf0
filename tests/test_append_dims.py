"""kv_append at every head dim: a group that migrates is cut into slices of tokens, each
taken by the threads of one channel pair each.

CPU: for every head dim the slices take each of the 32 tokens once and need no more threads
than there are. GPU: caches built by appends are byte for byte what kv_pack makes of all
tokens, with guarded rows behind the reserved ones.
"""
import os
import shutil
import subprocess
import textwrap

import pytest

from oracle import kvq_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_sparse_kv_gb300", "csrc")
DIMS = [32, 64, 96, 128, 160, 192, 224, 256]

_PROGRAM = textwrap.dedent(r"""
    #include <cstdio>
    #include "kvq_internal.h"
    int main() {
      for (int D = 32; D <= 256; D += 32) {
        const int pairs = D / 2, n = kvq::append_slices(D), each = 32 / n;
        int lowest = 99, highest = 0;
        for (int p = 0; p < pairs; ++p) {
          int taken[64] = {};
          for (int thread = 0; thread < kvq::kAppendThreads; ++thread)
            if (thread % pairs == p && thread / pairs < n)
              for (int t = 0; t < each; ++t) ++taken[thread / pairs * each + t];
          for (int t = 0; t < 64; ++t) {
            const int x = t < 32 ? taken[t] : 1 - taken[t];
            lowest = x < lowest ? x : lowest;
            highest = x > highest ? x : highest;
          }
        }
        std::printf("%d %d %d %d\n", D, n * pairs <= kvq::kAppendThreads, lowest, highest);
      }
      return 0;
    }
""")


def test_the_slices_take_every_token_once(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "slices.cu"
    src.write_text(_PROGRAM)
    exe = tmp_path / "slices"
    subprocess.run([nvcc, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert [tuple(map(int, x.split())) for x in out.splitlines()] == [(d, 1, 1, 1) for d in DIMS]


@pytest.mark.gpu
@pytest.mark.parametrize("win", ["bf16", "f32"])
@pytest.mark.parametrize("d", DIMS)
def test_appended_caches_are_packed_ones(d, win):
    torch = pytest.importorskip("torch")
    from quantized_sparse_kv_gb300 import kvq
    gen = torch.Generator(device="cuda").manual_seed(d)
    dt = torch.float32 if win == "f32" else torch.bfloat16
    k = torch.randn((2, 3, 260, d), generator=gen, device="cuda").to(dt)
    v = torch.randn((2, 3, 260, d), generator=gen, device="cuda").to(dt)
    cache = kvq.pack(k[:, :, :70], v[:, :, :70], 70, win, reserve=(9, 260))
    for x in (cache.k_codes, cache.v_codes):
        x.fill_(0xee)
    for x in (cache.k_scales, cache.v_scales):
        x.fill_(-1.0)
    for a, b in ((70, 71), (71, 200), (200, 201), (201, 260)):
        kvq.append(cache, k[:, :, a:b], v[:, :, a:b], 40)
    want = kvq.pack(k, v, cache.recent, win)
    assert cache.cut == 192
    got, ref = cache.used(), want.used()
    for name in got:
        assert torch.equal(got[name], ref[name]), name
    # what lies behind the groups is as it was
    assert bool((cache.k_codes[:, :, cache.gk:] == 0xee).all())
    assert bool((cache.v_codes[:, :, cache.cut:] == 0xee).all())
    assert bool((cache.k_scales[:, :, cache.gk:] == -1).all())
    assert bool((cache.v_scales[:, :, cache.cut:] == -1).all())
    host = O.pack(k.float().cpu().numpy(), v.float().cpu().numpy(), cache.recent, win)
    q = torch.randn((2, 6, 1, d), generator=gen, device="cuda")
    out = kvq.Attend(cache, q, out_dtype="f32").run()
    ref_out, _ = O.attend(q.cpu().numpy(), host)
    assert O.rel_l2(out.cpu().numpy(), ref_out) <= 1e-4  # (an fp32 kernel)
