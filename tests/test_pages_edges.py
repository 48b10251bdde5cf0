"""The paged cache at its ends: magnitudes and masks that strain the fp16 products, pools
and windows behind 32-bit offsets, many rows, waits that run out, and the bounds-checked
build. Tolerances as in test_pages.py.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kvq_oracle as O  # noqa: E402
from test_pages import (Model, TOL_F32, TOL_TENSOR, attention64, kvq, new_rows,  # noqa: E402,F401
                        poison, sequence_values)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def one_request(kvq, length, k, v, window, hk, d, wdt="bf16", page=64):  # noqa: F811
    """A cache with one request of these keys and values, and its host values."""
    pages = length // page + 2
    state = kvq.PageState(1, pages, page, pages, window)
    cache = kvq.PagedCache(state, hk, d, wdt)
    poison(cache)
    plan = kvq.page_tables(state, torch.tensor([length], device="cuda"), length)
    kvq.append_pages(cache, plan, k, v)
    assert kvq.read_status(plan.status) == 0
    model = Model(1, pages, page, pages, window)
    kept = [x.float().cpu().numpy() for x in (k, v)]
    return cache, sequence_values(model, [kept], 0, wdt)


def check_rows(kvq, cache, values, q, tol, heads=None):  # noqa: F811
    call = kvq.AttendPages(cache, q, torch.zeros(q.shape[0], dtype=torch.int32, device="cuda"),
                           out_dtype="f32")
    got = call.run().double().cpu().numpy()
    assert kvq.read_status(call.status) == 0
    for i in range(q.shape[0]):
        want = attention64(q[i].double().cpu().numpy(), *values)
        for h in range(q.shape[1]):
            assert O.rel_l2(got[i, h], want[h]) <= tol, (i, h)
    return call


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e-7, 1e-4, 0.02, 30.0, 5e3, 1e8])
def test_values_of_any_magnitude(kvq, d, size):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = 640
    k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    v = (torch.randn((n, 1, d), generator=gen, device="cuda") * size).bfloat16()
    cache, values = one_request(kvq, n, k, v, 0, 1, d)
    q = torch.randn((3, 8, d), generator=gen, device="cuda").bfloat16()
    check_rows(kvq, cache, values, q, TOL_TENSOR)


@pytest.mark.gpu
def test_magnitudes_that_change_along_a_request(kvq):  # noqa: F811
    # groups of large, small and zero values under scores that lie apart: the sum of the
    # probabilities keeps what the values do not show
    d, n = 128, 1024
    gen = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn((n, 2, d), generator=gen, device="cuda")
    v = torch.randn((n, 2, d), generator=gen, device="cuda")
    size = torch.ones(n, device="cuda")
    size[:320], size[320:352], size[352:640] = 1e-6, 0.0, 200.0
    size[700:800] = 1e5
    k[320:352] *= 3.0
    v *= size[:, None, None]
    k, v = k.bfloat16(), v.bfloat16()
    cache, values = one_request(kvq, n, k, v, 64, 2, d)
    q = torch.randn((4, 16, d), generator=gen, device="cuda").bfloat16()
    check_rows(kvq, cache, values, q, TOL_TENSOR)
    # zero values throughout, and a zero query
    cache, values = one_request(kvq, n, k, torch.zeros_like(v), 64, 2, d)
    out, _ = kvq.attend_pages(cache, q[:1], out_dtype="f32")
    assert bool((out == 0).all())
    cache, values = one_request(kvq, n, k, v, 64, 2, d)
    check_rows(kvq, cache, values, torch.zeros_like(q), TOL_TENSOR)


@pytest.mark.gpu
def test_a_key_far_above_the_others(kvq):  # noqa: F811
    # one key 10 nats above, with a zero value: the output is the others' (11 bits of P hold
    # down to 11.8 nats below the maximum)
    d, n = 128, 512
    gen = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn((1, 8, d), generator=gen, device="cuda")
    q = (q / q.norm(dim=-1, keepdim=True) * 2 + 0.5).bfloat16()
    mean = q.float().mean((0, 1))
    k = torch.randn((n, 1, d), generator=gen, device="cuda") * 0.3
    k[77, 0] += mean / (mean @ mean) * (10.0 * d ** 0.5)
    v = torch.randn((n, 1, d), generator=gen, device="cuda")
    v[77] = 0.0
    k, v = k.bfloat16(), v.bfloat16()
    cache, values = one_request(kvq, n, k, v, 0, 1, d)
    a = (values[0][0] @ q[0].double().cpu().numpy().T) / np.sqrt(d)
    gap = a[77] - np.median(a, axis=0)
    assert 6.0 < gap.min() and gap.max() < 11.8
    check_rows(kvq, cache, values, q, TOL_TENSOR)


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(128, "bf16"), (96, "f32")])
def test_nan_values_show_and_stay_where_they_are(kvq, d, wdt):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(6)
    state = kvq.PageState(2, 20, 32, 10, 32)
    cache = kvq.PagedCache(state, 2, d, wdt)
    poison(cache)
    k = torch.randn((300, 2, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((300, 2, d), generator=gen, device="cuda").bfloat16()
    v[199, 1, 5] = float("nan")   # the window of request 0, KV head 1, its last token
    k[299, 0, 3] = float("nan")   # the last key of request 1, KV head 0
    plan = kvq.page_tables(state, torch.tensor([200, 100], device="cuda"), 300)
    kvq.append_pages(cache, plan, k, v)
    q = torch.randn((4, 4, d), generator=gen, device="cuda").bfloat16()
    slot = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([199, 198, 99, 98], dtype=torch.int32, device="cuda")
    out, status = kvq.attend_pages(cache, q, slot, pos, out_dtype="f32")
    assert kvq.read_status(status) == 0
    bad = out.isnan()
    assert bool(bad[0, 2:, 5].all()) and not bool(bad[0, :2].any())
    assert not bool(bad[0, 2:, :5].any())
    assert not bool(bad[1].any()) and not bool(bad[3].any())
    assert bool(bad[2, :2].all()) and not bool(bad[2, 2:].any())


@pytest.mark.gpu
@pytest.mark.parametrize("wdt,d", [("bf16", 128), ("f32", 32)])
def test_pages_and_windows_behind_32_bits(kvq, wdt, d):  # noqa: F811
    # a pool and windows of more than 2^32 bytes; pages are taken from the end
    hk = 2
    rec = 40 * d * hk
    n_pages = (5 << 30) // rec
    window = 128
    tile = 64 * d * hk * 5 * (4 if wdt == "f32" else 2)
    slots = min(8192, (5 << 30) // tile + 1)
    window = 128 if slots * tile > 1 << 32 else 4000
    state = kvq.PageState(slots, n_pages, 32, 40, window)
    cache = kvq.PagedCache(state, hk, d, wdt)
    assert cache.pool.numel() > 1 << 32 and cache.ring.numel() > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(8)
    n = window + 400
    new = torch.zeros(slots, dtype=torch.int32, device="cuda")
    new[-1] = n
    k, kept_k = new_rows(gen, n, hk, d, torch.bfloat16, wdt)
    v, kept_v = new_rows(gen, n, hk, d, torch.bfloat16, wdt)
    plan = kvq.page_tables(state, new, n)
    kvq.append_pages(cache, plan, k, v)
    model = Model(1, 100, 32, 40, window)
    values = sequence_values(model, [[kept_k, kept_v]], 0, wdt)
    rows = torch.full((n,), slots - 1, dtype=torch.int32, device="cuda")
    got = kvq.page_values(cache, rows, torch.arange(n, device="cuda"), "f32")
    for x, want in zip(got, values):
        x = x.double().cpu().numpy().transpose(1, 0, 2)
        assert (np.abs(x - want) <= 2.0 ** -24 * np.abs(want)).all()
    q = torch.randn((1, 4, d), generator=gen, device="cuda").bfloat16()
    out, status = kvq.attend_pages(cache, q, rows[:1], out_dtype="f32")
    assert kvq.read_status(status) == 0
    want = attention64(q[0].double().cpu().numpy(), *values)
    assert O.rel_l2(out[0].double().cpu().numpy(), want) <= (TOL_TENSOR if wdt == "bf16" else TOL_F32)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 159, 161, 500, 3000])
def test_many_rows(kvq, rows):  # noqa: F811
    # rows of requests with 0 to 300 tokens, some of none, in any order
    rng = np.random.default_rng(rows)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    slots, d, window = 60, 64, 40
    state = kvq.PageState(slots, 500, 32, 20, window)
    cache = kvq.PagedCache(state, 1, d)
    poison(cache)
    lengths = [int(x) for x in rng.choice([0, 1, 31, 32, 72, 73, 104, 200, 300], slots)]
    total = sum(lengths)
    k, kept_k = new_rows(gen, total, 1, d, torch.bfloat16, "bf16")
    v, kept_v = new_rows(gen, total, 1, d, torch.bfloat16, "bf16")
    plan = kvq.page_tables(state, torch.tensor(lengths, device="cuda"), total)
    kvq.append_pages(cache, plan, k, v)
    model = Model(slots, 500, 32, 20, window)
    at = np.cumsum([0] + lengths)
    tokens = [[kept_k[a:b], kept_v[a:b]] for a, b in zip(at, at[1:])]
    slot = rng.integers(-1, slots, rows)
    q = torch.randn((rows, 3, d), generator=gen, device="cuda").bfloat16()
    out = torch.full(q.shape, 5.0, device="cuda")
    call = kvq.AttendPages(cache, q, torch.tensor(slot, device="cuda"), out=out)
    for _ in range(2):  # (the second run finds the first one's workspace)
        call.run()
        assert kvq.read_status(call.status) == 0 and call.path == "pages_tensor"
    got, q64 = out.double().cpu().numpy(), q.double().cpu().numpy()
    values = {}
    for i, s in enumerate(slot):
        if s < 0:
            assert (got[i] == 5.0).all()
        elif lengths[s] == 0:
            assert (got[i] == 0.0).all()
        else:
            if s not in values:
                values[s] = sequence_values(model, tokens, s, "bf16")
            assert O.rel_l2(got[i], attention64(q64[i], *values[s])) <= TOL_TENSOR, (i, s)


@pytest.mark.gpu
def test_runs_agree_to_the_last_bit(kvq):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(11)
    n, d = 20000, 128
    k = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    cache, _ = one_request(kvq, n, k, v, 100, 2, d)
    q = torch.randn((5, 16, d), generator=gen, device="cuda").bfloat16()
    rows = torch.zeros(5, dtype=torch.int32, device="cuda")
    call = kvq.AttendPages(cache, q, rows, out_dtype="f32")
    first = call.run().clone()
    for _ in range(5):
        assert torch.equal(call.run(), first)
    # the same row alone, or among others, is the same up to the order of the joins
    alone, _ = kvq.attend_pages(cache, q[:1], rows[:1], out_dtype="f32")
    assert O.rel_l2(alone[0].cpu().numpy(), first[0].cpu().numpy()) <= 1e-3


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported(kvq):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(12)
    n, d = 6000, 128
    k = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    cache, values = one_request(kvq, n, k, v, 128, 2, d)
    q = torch.randn((3, 16, d), generator=gen, device="cuda").bfloat16()
    rows = torch.zeros(3, dtype=torch.int32, device="cuda")
    call = kvq.AttendPages(cache, q, rows, out_dtype="f32")
    kvq.debug_set(20_000_000, 5)  # 20 ms; item 5 is never copied
    try:
        call.run()
        assert kvq.read_status(call.status) & kvq.DEV_TIMEOUT
    finally:
        kvq.debug_set(0, -1)
    call.status.zero_()
    check_rows(kvq, cache, values, q, TOL_TENSOR)
    got = call.run().double().cpu().numpy()
    assert kvq.read_status(call.status) == 0
    assert O.rel_l2(got[0], attention64(q[0].double().cpu().numpy(), *values)) <= TOL_TENSOR


@pytest.mark.gpu
def test_two_streams_at_once(kvq):  # noqa: F811
    """Two prepared calls over one cache, each with a workspace of its own."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    n, d = 9000, 128
    k = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    cache, values = one_request(kvq, n, k, v, 128, 2, d)
    q = torch.randn((2, 16, d), generator=gen, device="cuda").bfloat16()
    rows = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = [kvq.AttendPages(cache, q[i:i + 1], rows, out_dtype="f32") for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for i, c in enumerate(calls):
        assert int(c.status[0]) == 0
        want = attention64(q[i].double().cpu().numpy(), *values)
        assert O.rel_l2(c.out[0].double().cpu().numpy(), want) <= TOL_TENSOR


@pytest.mark.gpu
def test_both_builds_agree(tmp_path):
    from quantized_sparse_kv_gb300 import kvq as k
    files = []
    for lib in (k.LIB_PATH, k.DEBUG_LIB_PATH):
        out = str(tmp_path / (os.path.basename(lib) + ".npz"))
        r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_pages_cases.py"),
                            lib, out], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
        files.append(np.load(out))
    rel, dbg = files
    assert int(rel["checks"]) == 0 and int(dbg["checks"]) == 1
    assert set(rel.files) == set(dbg.files)
    for name in rel.files:
        if name == "checks":
            continue
        if name.startswith("status_"):
            assert int(rel[name]) == 0 and int(dbg[name]) == 0, name
        else:
            assert rel[name].tobytes() == dbg[name].tobytes(), name


@pytest.mark.gpu
def test_waits_that_run_out_at_any_item_end_the_call(kvq):  # noqa: F811
    # slices of several units each, whose ends are where the warps of a CTA meet
    gen = torch.Generator(device="cuda").manual_seed(14)
    d, rows = 64, 3000
    k = torch.randn((150, 1, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((150, 1, d), generator=gen, device="cuda").bfloat16()
    cache, values = one_request(kvq, 150, k, v, 40, 1, d)
    q = torch.randn((rows, 3, d), generator=gen, device="cuda").bfloat16()
    call = kvq.AttendPages(cache, q, torch.zeros(rows, dtype=torch.int32, device="cuda"),
                           out_dtype="f32")
    for item in [*range(24), 3 * rows - 1]:
        kvq.debug_set(2_000_000, item)  # 2 ms
        try:
            call.run()
            assert kvq.read_status(call.status) & kvq.DEV_TIMEOUT
        finally:
            kvq.debug_set(0, -1)
        call.status.zero_()
    got = call.run()
    assert kvq.read_status(call.status) == 0
    for i in (0, 1, rows - 1):
        want = attention64(q[i].double().cpu().numpy(), *values)
        assert O.rel_l2(got[i].double().cpu().numpy(), want) <= TOL_TENSOR


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("rows,group", [(2, 1), (2, 11), (700, 3)])
def test_the_fp32_kernel_at_every_head_dim(kvq, d, rows, group):  # noqa: F811
    # few rows share a request's groups among CTAs, many have one each; the last row of a
    # request is NaN and is attended by the first query row alone
    gen = torch.Generator(device="cuda").manual_seed(d + rows)
    n = 391
    k = torch.randn((n, 2, d), generator=gen, device="cuda")
    v = torch.randn((n, 2, d), generator=gen, device="cuda")
    v[n - 1] = float("nan")
    cache, (kk, vv) = one_request(kvq, n, k, v, 50, 2, d, "f32", 32)
    q = torch.randn((rows, 2 * group, d), generator=gen, device="cuda")
    pos = torch.randint(0, n - 1, (rows,), generator=gen, device="cuda").int()
    pos[0], pos[1] = n - 1, n - 2
    slot = torch.zeros(rows, dtype=torch.int32, device="cuda")
    call = kvq.AttendPages(cache, q, slot, pos)
    got = call.run().double().cpu().numpy()
    assert kvq.read_status(call.status) == 0 and call.path == "pages_rows"
    assert np.isnan(got[0]).all() and not np.isnan(got[1:]).any()
    for i in {1, rows // 2, rows - 1}:
        p = int(pos[i]) + 1
        want = attention64(q[i].double().cpu().numpy(), kk[:, :p], vv[:, :p])
        assert O.rel_l2(got[i], want) <= TOL_F32
