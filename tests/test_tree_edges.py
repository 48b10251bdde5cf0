"""kv_attend_tree: hand-overs of short segments, one key far above a long flat tail
(tolerances as in test_tree.py)."""
import math

import pytest
import torch

from test_tree import (TOL_F32, TOL_TENSOR, ancestors, compare, dequant, inputs,  # noqa: F401 (fixture)
                       kvq, make, plain, random_tree)


@pytest.mark.gpu
@pytest.mark.parametrize("b,g,n,recent,t", [(250, 8, 100, 100, 5), (1000, 4, 60, 60, 1),
                                            (400, 8, 90, 0, 3), (170, 8, 100, 64, 16)])
def test_many_short_units_agree(kvq, b, g, n, recent, t):  # noqa: F811
    """Shared rows and one or two tiles a unit, several units a CTA: MMA warps without a step
    in a unit keep up with the others, run after run."""
    c = make(kvq, b, 2, n, 128, recent)
    q, k, v = inputs(b, 2 * g, 2, t, 128)
    par = random_tree(b, t, n + t)
    call = kvq.AttendTree(c, q, k, v, par, out_dtype="f32")
    first = call.run().clone()
    assert kvq.read_status(call.status) == 0 and call.path == "tree_tensor"
    compare(first, plain(c, kvq, q, k, v, par), par, TOL_TENSOR)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        differ += (call.run() != first).any()
    assert int(differ) == 0 and kvq.read_status(call.status) == 0


def one_key_over_a_flat_tail(kvq, b, n, nats):  # noqa: F811
    """A cache whose first key stands `nats` above the others, which are all equal, with V = 0
    there: the output is the tail's sum of V over 2^s + tail. Scores are exact (key 0.875 =
    7 * 0.125, log2 scale 2^-3, q a bf16 number): s = 128 * 0.875 * q / 8 = 14 q."""
    k = torch.zeros((b, 2, n, 128), device="cuda", dtype=torch.bfloat16)
    k[:, :, 0] = 0.875
    g = torch.Generator(device="cuda").manual_seed(5)
    v = (1.0 + 0.5 * torch.randn((b, 2, n, 128), generator=g, device="cuda")).bfloat16()
    v[:, :, 0] = 0.0
    c = kvq.pack(k, v, 0, "bf16")
    q = torch.tensor(nats / math.log(2.0) / 14.0).bfloat16().item()
    return c, q, 2.0 ** (14.0 * q)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nats", [8.0, 12.0, 14.0, 15.0, 16.0, 17.0])
@pytest.mark.parametrize("t", [1, 32])
def test_a_key_far_above_a_flat_tail(kvq, dt, nats, t):  # noqa: F811
    """P is rounded to fp16 against a reference 2^9 below the row's maximum: at 17 nats the tail's
    P is 2.1e-5, off by 2^-25 / 2.1e-5 = 1.4e-3 of itself at most. With the values' 2^-11 (twice)
    that stays below 5e-3. The first key's slice holds most of its unit's tail."""
    b, n = 80 if dt == torch.bfloat16 else 2, 2048
    c, x, first = one_key_over_a_flat_tail(kvq, b, n, nats)
    q = torch.full((b, 16, t, 128), x, device="cuda").to(dt)
    kt = torch.zeros((b, 2, t, 128), device="cuda").to(dt)
    vt = torch.ones((b, 2, t, 128), device="cuda").to(dt)
    par = torch.full((b, t), -1, dtype=torch.int32, device="cuda")  # each sees itself alone
    call = kvq.AttendTree(c, q, kt, vt, par, sm_scale=math.log(2.0) / 8.0, out_dtype="f32")
    out = call.run()
    assert kvq.read_status(call.status) == 0
    _, v = dequant(c, kvq)
    want = ((v.sum(2) + 1.0) / (first + n)).repeat_interleave(8, 1).unsqueeze(2)  # (the key itself: 1)
    want = want.expand(out.shape)
    tol = TOL_TENSOR if dt == torch.bfloat16 else TOL_F32
    assert float((out.double() - want).norm() / want.norm()) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,n,t", [(1, 3000, 1), (2, 700, 5), (2, 700, 40), (24, 260, 20)])
def test_a_nan_query_row_is_nan_and_stays_alone(kvq, dt, b, n, t):  # noqa: F811
    """Over one partial and several, shared rows and two groups of them. (The NaN row's warp takes
    its maxima every step, which moves its neighbours' references: within the tolerance.)"""
    c = make(kvq, b, 2, n, 128, 70)
    q, k, v = inputs(b, 16, 2, t, 128, dt)
    par = random_tree(b, t, 7)
    want = plain(c, kvq, q, k, v, par)
    q[-1, 3, t - 1, 17] = torch.nan
    call = kvq.AttendTree(c, q, k, v, par, out_dtype="f32")
    out = call.run()
    assert kvq.read_status(call.status) == 0
    assert bool(torch.isnan(out[-1, 3, t - 1]).all())
    out[-1, 3, t - 1], want[-1, 3, t - 1] = 0.0, 0.0
    compare(out, want, par, TOL_TENSOR if dt == torch.bfloat16 else TOL_F32)


BEYOND = [65536.0, -1e5, 3e38, float("inf"), float("-inf"), float("nan")]


@pytest.mark.gpu
@pytest.mark.parametrize("x", BEYOND)
@pytest.mark.parametrize("t", [3, 40])
def test_elements_beyond_fp16_show(kvq, x, t):  # noqa: F811
    """The tensor-core kernel's operands end at 65,504: what lies beyond makes the rows that see
    it NaN or infinite, instead of counting as some finite number, and no other row."""
    b, n, recent = 2, 500, 70
    q, k, v = inputs(b, 16, 2, t, 128)
    par = random_tree(b, t, 11)
    seen = ancestors(par)
    clean = make(kvq, b, 2, n, 128, recent)
    want = plain(clean, kvq, q, k, v, par)

    def run(c=clean, q=q, k=k, v=v):
        call = kvq.AttendTree(c, q, k, v, par, out_dtype="f32")
        out = call.run()
        assert kvq.read_status(call.status) == 0 and call.path == "tree_tensor"
        return out

    def check(out, odd):  # the odd elements are not finite, the rest is what it was
        assert not bool(torch.isfinite(out[odd]).any())
        compare(torch.where(odd, 0.0, out), torch.where(odd, 0.0, want), par, TOL_TENSOR)
    none = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    odd = none.clone()
    odd[1, 4, t - 1] = True
    q2 = q.clone()
    q2[1, 4, t - 1, 100] = x
    check(run(q=q2), odd)
    sees = seen[1, :, 1]                                     # rows of sequence 1 that see token 1
    odd = none.clone()
    odd[1, 8:, sees] = True
    k2 = k.clone()
    k2[1, 1, 1, 7] = x
    check(run(k=k2), odd)
    odd = none.clone()
    odd[1, 8:, sees, 77] = True
    v2 = v.clone()
    v2[1, 1, 1, 77] = x
    out = run(v=v2)
    check(out, odd)
    if not math.isnan(x):
        assert bool((out[odd] == math.copysign(math.inf, x)).all())
    c = make(kvq, b, 2, n, 128, recent)
    c.k_window[0, 1, recent - 1, 3] = x
    odd = none.clone()
    odd[0, 8:] = True
    check(run(c=c), odd)
    c = make(kvq, b, 2, n, 128, recent)
    c.v_window[0, 1, 0, 3] = x
    odd = none.clone()
    odd[0, 8:, :, 3] = True
    check(run(c=c), odd)


@pytest.mark.gpu
def test_the_largest_fp16_elements_are_exact(kvq):  # noqa: F811
    """65,280 is bf16's last number below 2^16: values that large are what they are."""
    b, n, t = 1, 90, 4
    c = make(kvq, b, 1, n, 128, 90)
    q, k, v = inputs(b, 8, 1, t, 128)
    par = random_tree(b, t, 2)
    v[..., 5] = 65280.0
    c.v_window[..., 5] = 65280.0
    c.v_window[..., 6] = -65280.0
    out, st = kvq.attend_tree(c, q, k, v, par, out_dtype="f32")
    assert kvq.read_status(st) == 0
    compare(out, plain(c, kvq, q, k, v, par), par, TOL_TENSOR)
    assert bool(((out[..., 5] / 65280.0 - 1).abs() <= 2.0 ** -10).all())
