"""kv_rope: rotary positions.

CPU: the frequency table against the formulas in Python floats, and every
refusal. GPU: the rotation against a 64-bit plain form. Tolerances, per
element of a pair (x0, x1) rotated with amplitude a: the phase is exact to
2^-24 of itself (at most 2^-24 * pi radians), sincospif is within 2 units of
2^-23, the amplitude and the two products and their sum round four times at
2^-24; together below 8e-7 * a * (|x0| + |x1|), taken as 1e-6. The frequency
itself is a 64-bit float on both sides (each a few roundings of 2^-53), so two
evaluations of the angle pos * f may differ by 2^-50 of it. A bf16 result adds
its own rounding, 2^-8 of the value.
"""
import ctypes
import math

import pytest
import torch

ADDR = ctypes.c_void_p(1 << 20)   # aligned placeholder, never dereferenced
SCALINGS = {
    "none": dict(), "linear": dict(factor=2.5), "base": dict(factor=8.0),
    "ramp": dict(factor=16.0, original=4096, fast=32.0, slow=1.0),
    "bands": dict(factor=8.0, original=8192, low=1.0, high=4.0),
}


@pytest.fixture(scope="module")
def kvq():
    import os
    from quantized_sparse_kv_gb300 import build, kvq as k
    if not os.path.exists(k.LIB_PATH):
        build.build()
    k.load_library()
    return k


def frequencies(r, base, scaling):
    """Angular frequencies and amplitude from the header's formulas."""
    s = SCALINGS[scaling]
    if scaling == "base":
        base = base * s["factor"] ** (r / (r - 2))
    f = [base ** (-2 * i / r) for i in range(r // 2)]
    amp = 1.0
    if scaling == "linear":
        f = [x / s["factor"] for x in f]
    if scaling == "ramp":
        def x_of(t):
            return r * math.log(s["original"] / (2 * math.pi * t)) / (2 * math.log(base))
        lo = max(0, math.floor(x_of(s["fast"])))
        hi = min(r - 1, math.ceil(x_of(s["slow"])))
        w = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(r // 2)]
        f = [x * (1 - u) + x / s["factor"] * u for x, u in zip(f, w)]
        amp = 0.1 * math.log(s["factor"]) + 1
    if scaling == "bands":
        w = [min(1.0, max(0.0, (s["original"] * x / (2 * math.pi) - s["low"]) /
                          (s["high"] - s["low"]))) for x in f]
        f = [x * u + x / s["factor"] * (1 - u) for x, u in zip(f, w)]
    return f, amp


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("r,base", [(128, 10000.0), (64, 500000.0), (30, 10000.0)])
def test_turns_follow_the_formulas(kvq, scaling, r, base):
    plan = kvq.RopePlan(r, base=base, scaling=scaling, device="cpu", **SCALINGS[scaling])
    f, amp = frequencies(r, base, scaling)
    for t, x in zip(plan.turns_host, f):
        assert t / 2.0 ** 64 == pytest.approx(x / (2 * math.pi), rel=1e-14)
    assert plan.amplitude == pytest.approx(amp, rel=1e-6)


def test_turns_refusals(kvq):
    lib = kvq.load_library()
    out = (ctypes.c_uint64 * 128)()
    amp = ctypes.c_float()

    def call(r=64, base=10000.0, sc=None):
        s = kvq.KvqRopeScaling(*sc) if sc else None
        return lib.kvq_rope_turns(r, base, ctypes.byref(s) if s else None, out, ctypes.byref(amp))
    assert call() == 0
    for r in (0, -2, 3, 258):
        assert call(r=r) == 1
    for base in (1.0, 0.0, float("nan"), float("inf")):
        assert call(base=base) == 1
    assert call(sc=(9, 2.0, 0.0, 0.0, 0.0)) == 1             # unknown kind
    assert call(sc=(1, 0.5, 0.0, 0.0, 0.0)) == 1             # factor below 1
    assert call(sc=(1, float("nan"), 0.0, 0.0, 0.0)) == 1
    assert call(r=2, sc=(2, 2.0, 0.0, 0.0, 0.0)) == 1        # base scaling of one pair
    assert call(sc=(3, 2.0, 4096.0, 1.0, 32.0)) == 1         # ramp limits reversed
    assert call(sc=(3, 2.0, 0.0, 32.0, 1.0)) == 1            # no original context
    assert call(sc=(4, 2.0, 4096.0, 4.0, 1.0)) == 1          # band limits reversed
    assert call(sc=(4, 2.0, 4096.0, 1.0, 4.0)) == 0
    with pytest.raises(TypeError):
        kvq.RopePlan(64, scaling="ramp", factor=2.0, device="cpu")
    with pytest.raises(ValueError):
        kvq.RopePlan(64, layout="other", device="cpu")


def test_ramp_outside_the_pairs(kvq):
    """A ramp that lies past the last pair leaves every frequency alone, one before
    the first pair scales all but that one (both ends are clamped to the pairs)."""
    r, base, factor = 64, 10.0, 4.0

    def turns(original):
        out, amp = (ctypes.c_uint64 * (r // 2))(), ctypes.c_float()
        sc = kvq.KvqRopeScaling(3, factor, original, 32.0, 1.0)
        assert kvq.load_library().kvq_rope_turns(r, base, ctypes.byref(sc), out,
                                                 ctypes.byref(amp)) == 0
        return [x / 2.0 ** 64 * 2 * math.pi for x in out]

    plain = [base ** (-2.0 * i / r) for i in range(r // 2)]
    # x(32) = 64 ln(original / 201) / (2 ln 10) is above 63 from about 19,000 on
    for got, want in zip(turns(1e6), plain):
        assert abs(got - want) <= 1e-14 * want
    # x(1) is below 0 up to 6 tokens
    short = turns(4.0)
    assert abs(short[0] - plain[0]) <= 1e-14
    for got, want in zip(short[1:], plain[1:]):
        assert abs(got - want / factor) <= 1e-14 * want


def test_call_refusals(kvq):
    lib = kvq.load_library()

    def call(n_tensors=1, dtype=1, batch=2, n=3, d=128, rot=128, layout=0, amp=1.0, turns=ADDR,
             pos=ADDR, heads=2, inp=ADDR, strides=(768, 384, 128)):
        t = (kvq.KvqRopeTensor * 3)(*[kvq.KvqRopeTensor(inp, ADDR, heads, 1, *strides)] * 3)
        return lib.kv_rope(t, n_tensors, dtype, batch, n, d, rot, layout, turns, amp, 0, pos, None,
                           None)
    assert call(n=0) == 0 and call(batch=0) == 0 and call(n=0, pos=None) == 0
    for kw in (dict(n_tensors=0), dict(n_tensors=4), dict(dtype=2), dict(batch=-1), dict(n=-1),
               dict(d=100), dict(d=288), dict(rot=0), dict(rot=63), dict(rot=130),
               dict(layout=2), dict(amp=0.0), dict(amp=float("nan")), dict(turns=None),
               dict(pos=None), dict(heads=0), dict(inp=None), dict(strides=(-8, 8, 8))):
        assert call(**kw) == 1, kw
    for kw in (dict(turns=ctypes.c_void_p((1 << 20) + 8)), dict(inp=ctypes.c_void_p((1 << 20) + 2)),
               dict(strides=(768, 384, 132)), dict(dtype=0, strides=(768, 384, 130))):
        assert call(**kw) == 2, kw
    assert call(batch=1 << 16, n=1 << 16) == 3


# ------------------------------------------------------------------ GPU


def plain(x, pos, plan_args, r, layout, inverse):
    f, amp = frequencies(r, *plan_args)
    ang = pos.double()[:, None, :, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = ang.cos() * amp, ang.sin() * amp * (-1 if inverse else 1)
    y = x.double().clone()
    i0, i1 = ((slice(0, r // 2), slice(r // 2, r)) if layout == "half"
              else (slice(0, r, 2), slice(1, r, 2)))
    a, b = x.double()[..., i0], x.double()[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    bound = torch.zeros_like(y)
    bound[..., i0] = bound[..., i1] = (1e-6 + 2.0 ** -50 * ang.abs()) * amp * (a.abs() + b.abs())
    return y, bound


def check(out, x, pos, plan_args, r, layout, inverse):
    y, bound = plain(x, pos, plan_args, r, layout, inverse)
    if x.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * y.abs()
    assert out.is_contiguous() and out.dtype == x.dtype
    err = (out.double() - y).abs()
    assert bool((err <= bound + 1e-30).all()), float((err - bound).max())
    assert torch.equal(out[..., r:], x[..., r:])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (32, 2), (32, 32), (64, 30), (256, 256),
                                 (96, 48), (160, 158)])
def test_rotation(kvq, layout, dtype, d, r):
    g = torch.Generator(device="cuda").manual_seed(d * 1000 + r)
    for b, n, hq, hk, scaling in ((1, 1, 1, 1, "none"), (3, 5, 4, 2, "ramp"), (2, 131, 7, 1, "bands")):
        q = torch.randn((b, hq, n, d), generator=g, device="cuda").to(dtype)
        k = torch.randn((b, hk, n, d), generator=g, device="cuda").to(dtype)
        pos = torch.randint(-(1 << 31), (1 << 31) - 1, (b, n), generator=g, device="cuda")
        pos[0, 0] = 0
        pos[-1, -1] = (1 << 31) - 1
        if n > 4:  # ordinary positions among the far ones
            pos[:, 1:4] = torch.tensor([1, -1, 32767], device="cuda")
        plan = kvq.RopePlan(r, layout=layout, scaling=scaling, **SCALINGS[scaling])
        for inverse in (False, True):
            oq, ok = kvq.rope(plan, q, k, pos, inverse=inverse)
            torch.cuda.synchronize()
            check(oq, q, pos, (10000.0, scaling), r, layout, inverse)
            check(ok, k, pos, (10000.0, scaling), r, layout, inverse)


@pytest.mark.gpu
@pytest.mark.parametrize("layout,r", [("half", 128), ("half", 64), ("interleaved", 128),
                                      ("half", 36)])
def test_projection_rows_in_place_and_misaligned(kvq, layout, r):
    g = torch.Generator(device="cuda").manual_seed(r)
    b, n, hq, hk, d = 2, 37, 6, 2, 128
    rows = torch.randn((b, n, hq + 2 * hk, d), generator=g, device="cuda").bfloat16()
    q, k, v = (rows[:, :, i:j].transpose(1, 2) for i, j in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    pos = torch.randint(0, 1 << 20, (b, n), generator=g, device="cuda")
    plan = kvq.RopePlan(r, layout=layout)
    call = kvq.Rope(plan, q, k, pos, v=v)
    assert not [x for x in call._copies if x[0].dtype == torch.bfloat16]  # rows are read in place
    oq, ok, ov = call.run()
    check(oq, q, pos, (10000.0, "none"), r, layout, False)
    check(ok, k, pos, (10000.0, "none"), r, layout, False)
    assert torch.equal(ov, v) and ov.is_contiguous()
    # a prepared call sees new contents of its inputs, copied ones included
    rows.neg_()
    pos.add_(5)
    call.run()
    check(oq, q, pos, (10000.0, "none"), r, layout, False)
    # rows that do not start on 16 bytes, and a broadcast batch
    odd = torch.randn((b, hq, n, d + 1), generator=g, device="cuda").bfloat16()[..., 1:]
    one = torch.randn((1, hk, n, d), generator=g, device="cuda").bfloat16().expand(b, hk, n, d)
    oq, ok = kvq.rope(plan, odd, one, pos)
    check(oq, odd, pos, (10000.0, "none"), r, layout, False)
    check(ok, one, pos, (10000.0, "none"), r, layout, False)
    # in place
    x = q.contiguous()
    want = kvq.rope(plan, x, None, pos)[0]
    kvq.Rope(plan, x, None, pos, out=[x]).run()
    assert torch.equal(x, want)


@pytest.mark.gpu
def test_gradient(kvq):
    # the call is linear, so its gradient is its transpose: against autograd through the plain
    # formula, and against differences, which are exact for a linear map up to rounding
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((2, 3, 9, 64), generator=g, device="cuda")
    gy = torch.randn_like(x)
    pos = torch.randint(0, 5000, (2, 9), generator=g, device="cuda")
    for layout, scaling in (("half", "ramp"), ("interleaved", "none")):
        plan = kvq.RopePlan(48, layout=layout, scaling=scaling, **SCALINGS[scaling])
        gx = kvq.rope(plan, gy, None, pos, inverse=True)[0]
        f, amp = frequencies(48, 10000.0, scaling)
        xx = x.double().requires_grad_()
        ang = pos.double()[:, None, :, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
        a, b = ((xx[..., :24], xx[..., 24:48]) if layout == "half"
                else (xx[..., 0:48:2], xx[..., 1:48:2]))
        y0, y1 = a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()
        rot = (torch.cat((y0, y1), -1) if layout == "half"
               else torch.stack((y0, y1), -1).flatten(-2)) * amp
        y = torch.cat((rot, xx[..., 48:]), -1)
        (want,) = torch.autograd.grad(y, xx, gy.double())
        # 1e-6 a (|g0| + |g1|), both below 6
        assert float((gx.double() - want).abs().max()) <= 1.2e-5 * amp
        e = torch.randn_like(x)
        up = kvq.rope(plan, x + e, None, pos)[0].double()
        dn = kvq.rope(plan, x - e, None, pos)[0].double()
        diff = float(((up - dn) / 2 * gy.double()).sum())
        assert diff == pytest.approx(float((gx.double() * e.double()).sum()), abs=2e-3)


@pytest.mark.gpu
def test_captured_and_on_another_stream(kvq):
    q = torch.randn((2, 4, 3, 128), device="cuda").bfloat16()
    k = torch.randn((2, 2, 3, 128), device="cuda").bfloat16()
    pos = torch.arange(6, device="cuda", dtype=torch.int32).view(2, 3)
    plan = kvq.RopePlan(128)
    call = kvq.Rope(plan, q, k, pos)
    want = [x.clone() for x in call.run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call.run()
    for o in call.out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(call.out, want))
    pos.add_(7)  # a replay reads the new positions
    graph.replay()
    torch.cuda.synchronize()
    check(call.out[0], q, pos, (10000.0, "none"), 128, "half", False)
