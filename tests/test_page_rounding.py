"""The division-free int4 codes of fp32 values in kv_append_pages, on the CPU.

int4_round.cuh is compiled as a host program: wherever code8_clear answers true its code
equals clamp(rint(fl(x / s)), -7, 7), s = fl(amax / 7), on random values of every
magnitude, on values next to halfway between two codes (the nearest floats to (k + 1/2) s
and a few steps to either side) and at the ends; and it answers true for nearly all of
the random ones.
"""
import os
import shutil
import subprocess
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_sparse_kv_gb300", "csrc")

_PROGRAM = textwrap.dedent(r"""
    #include <cstdio>
    #include <cmath>
    #include <random>
    #include "int4_round.cuh"
    static long clear = 0, bad = 0, near_clear = 0;
    static bool check(float x, float amax) {
      if (std::fabs(x) > amax) return false;
      const float s = amax / 7.0f, r = kvq::recip_of(s);
      uint32_t c;
      if (!kvq::code8_clear(x, r, c)) return false;
      int want = 8;
      if (s != 0.0f) {
        float w = std::nearbyint(x / s);
        want = 8 + static_cast<int>(w > 7.0f ? 7.0f : w < -7.0f ? -7.0f : w);
      }
      if (static_cast<int>(c & 0xffu) != want) ++bad;
      return true;
    }
    int main() {
      std::mt19937_64 gen(1);
      std::uniform_real_distribution<float> u(-1.0f, 1.0f);
      long all = 0, ties = 0;
      for (int e = -100; e <= 127; ++e) {
        for (int i = 0; i < 20000; ++i) {
          const float amax = std::ldexp(1.0f + std::fabs(u(gen)), e - (e == 127));
          if (!kvq::recip_ok(amax)) continue;
          ++all;
          clear += check(u(gen) * amax, amax);
          check(amax, amax);
          check(-amax, amax);
          check(0.0f, amax);
          if (i >= 500) continue;
          for (int k = -7; k < 7; ++k) {
            float x = (k + 0.5f) * (amax / 7.0f);
            for (int d = 0; d < 24; ++d) x = std::nextafter(x, -INFINITY);
            for (int d = 0; d < 48; ++d, x = std::nextafter(x, INFINITY)) {
              ++ties;
              near_clear += check(x, amax);
            }
          }
        }
      }
      clear += check(0.0f, 0.0f);
      uint32_t c;
      std::printf("%ld %ld %ld %ld %ld %d\n", all, clear, ties, near_clear, bad,
                  static_cast<int>(kvq::code8_clear(1.0f, NAN, c)));
      return 0;
    }
""")


def test_clear_codes_are_those_of_the_division(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "clear_check.cu"
    src.write_text(_PROGRAM)
    exe = tmp_path / "clear_check"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-Xcompiler", "-ffp-contract=off", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    every, clear, ties, near_clear, bad, nan = map(int, out)
    assert every > 4 * 10 ** 6 and ties > 7 * 10 ** 7
    assert bad == 0 and nan == 0
    assert clear > 0.999 * every
    assert near_clear < ties
