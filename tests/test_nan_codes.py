"""A NaN among the values that become int4 codes leaves the other codes what they are
without it (the rule of kv_pack: the code of a NaN is unspecified, the others' are not, and a
NaN does not enter amax).

CPU: int4_round.cuh as a host program, whose sums give a NaN the bits the device gives it:
in every pair of a NaN and a value, the value's nibble is clamp(rint(fl(x / s)), -7, 7) + 8 and
the NaN's is a code. GPU: kv_pack, kv_append and kv_append_pages on values with NaNs at even
and odd channels of K, at tokens t and t + 8 of V and in whole runs, against the same values
with zeros in the NaNs' places (which leave amax as it is too).
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
    #include "int4_round.cuh"
    static float bf16(uint32_t h) { uint32_t u = h << 16; float f; memcpy(&f, &u, 4); return f; }
    static uint32_t want(float x, float s) {
      if (s == 0.0f) return 8;
      const float c = std::nearbyint(x / s);
      return static_cast<uint32_t>(8 + static_cast<int>(c > 7.0f ? 7.0f : c < -7.0f ? -7.0f : c));
    }
    int main() {
      long pairs = 0, bad = 0, outside = 0;
      const uint32_t nans[] = {0x7fc0, 0x7f81, 0x7fff, 0xffc0, 0xff81, 0xffff};
      for (int ha = 0; ha < 0x7f80; ha += 37) {
        const float amax = bf16(ha);
        if (!kvq::recip_ok(amax)) continue;
        const float s = kvq::scale_recip(amax), r = kvq::recip_of(s);
        const uint64_t ns = kvq::pair64(-s, -s), rr = kvq::pair64(r, r);
        for (int hx = 0; hx <= ha; hx += ha - hx < 64 ? 1 : 97) {
          for (int sg = 0; sg < 2; ++sg) {
            const uint32_t x = (hx | (sg << 15)) << 16;
            const uint32_t c = want(sg ? -bf16(hx) : bf16(hx), s);
            pairs += 2;
            if ((kvq::code_byte_pair(x, x, ns, rr) & 0xffu) != c * 17u) ++bad;
            for (uint32_t n : nans) {
              const uint32_t a = kvq::code_byte_pair(n << 16, x, ns, rr) & 0xffu;
              const uint32_t b = kvq::code_byte_pair(x, n << 16, ns, rr) & 0xffu;
              if (a >> 4 != c || (b & 15u) != c) ++bad;
              if ((a & 15u) == 0 || b >> 4 == 0) ++outside;
            }
          }
        }
      }
      std::printf("%ld %ld %ld\n", pairs, bad, outside);
      return 0;
    }
""")


def test_a_nan_leaves_the_other_nibble(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "nan_check.cu"
    src.write_text(_PROGRAM)
    exe = tmp_path / "nan_check"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-Xcompiler", "-ffp-contract=off", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    pairs, bad, outside = map(int, out)
    assert pairs > 10 ** 5 and (bad, outside) == (0, 0)


def values_with_nans(tokens, heads, d, dt, tokens_first):
    """k, v with NaNs and with zeros in their places, and where they are."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(tokens + d)
    out = []
    for _ in range(2):
        x = torch.randn((tokens, heads, d), generator=gen, device="cuda").to(dt)
        at = torch.rand(x.shape, generator=gen, device="cuda") < 0.01
        at[0, 0, 0::2] = True       # the even channels of a token, then the odd ones
        at[1, 0, 1::2] = True
        at[32:40, heads - 1, 5] = True    # tokens t, and further on t + 8
        at[72:80, heads - 1, 6] = True
        at[96:128, 0, 4] = True     # a group of a channel without any number
        at[100, 0, :32] = True      # 32 features without any number
        out.append((x, at))
    k, v = ((x.masked_fill(at, float("nan")), x.masked_fill(at, 0.0), at) for x, at in out)
    if not tokens_first:
        k, v = ([y.transpose(0, 1)[None].contiguous() for y in x] for x in (k, v))
    return k, v


def nibbles(codes):
    import torch
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def check_cache(got, want, at_k, at_v):
    """Two packed caches agree in all codes and scales but the codes of the NaNs."""
    import torch
    a, b = got.used(), want.used()
    cut = got.cut
    assert cut >= 128
    assert torch.equal(a["k_scales"], b["k_scales"]) and torch.equal(a["v_scales"], b["v_scales"])
    for name, at in (("k_codes", at_k), ("v_codes", at_v)):
        x, y = (nibbles(c[name]).reshape(*at.shape[:2], -1, at.shape[3])[:, :, :cut] for c in (a, b))
        where = at[:, :, :cut]
        assert int(where.sum()) > 100
        assert torch.equal(x.masked_fill(where, 0), y.masked_fill(where, 0)), name
        assert int(x.min()) >= 1 and int(x.max()) <= 15


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_pack_and_append_around_nans(d, dt):
    torch = pytest.importorskip("torch")
    from quantized_sparse_kv_gb300 import kvq
    dt = getattr(torch, dt)
    k, v = values_with_nans(256, 2, d, dt, False)
    win = "f32" if dt == torch.float32 else "bf16"
    caches = [kvq.pack(k[i], v[i], 64, win) for i in range(2)]
    check_cache(*caches, k[2], v[2])
    caches = []
    for i in range(2):
        c = kvq.pack(k[i][:, :, :40], v[i][:, :, :40], 40, win, reserve=(8, 300))
        kvq.append(c, k[i][:, :, 40:], v[i][:, :, 40:], 32)
        caches.append(c)
    check_cache(*caches, k[2], v[2])


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("steps", [[256], [1] * 40 + [100, 1, 115]])
def test_append_pages_around_nans(d, wdt, steps):
    torch = pytest.importorskip("torch")
    from quantized_sparse_kv_gb300 import kvq
    dt = torch.float32 if wdt == "f32" else torch.bfloat16
    k, v = values_with_nans(256, 2, d, dt, True)
    got = []
    for i in range(2):
        state = kvq.PageState(1, 8, 64, 8, 32)
        cache = kvq.PagedCache(state, 2, d, wdt)
        first = 0
        for n in steps:
            plan = kvq.page_tables(state, torch.tensor([n], device="cuda"), n)
            kvq.append_pages(cache, plan, k[i][first:first + n], v[i][first:first + n])
            assert kvq.read_status(plan.status) == 0
            first += n
        rows = torch.zeros(256, dtype=torch.int32, device="cuda")
        got.append(kvq.page_values(cache, rows, torch.arange(256, device="cuda"), "f32"))
    for x, y, at in zip(got[0], got[1], (k[2], v[2])):
        cut = state.cut(256)
        assert int(at[:cut].sum()) > 100
        assert torch.equal(x.masked_fill(at, 0.0), y.masked_fill(at, 0.0))
        assert bool(x[cut:][at[cut:]].isnan().all()) and not bool(x[:cut].isnan().any())
