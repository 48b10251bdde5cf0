"""kv_attend_tree: drafted tokens over the cache and their ancestors.

CPU: refusals and kernel choice through the workspace query. GPU: against a
plain form in 64 bits on the dequantized cache. Tolerances: the fp32 kernel's
relative L2 is held to 1e-5, as the other fp32 paths. The tensor-core kernel
rounds each int4 key and value twice to fp16 (scale, product; 2^-11 relative at
most each, rms 2^-11 / sqrt(3) = 2.8e-4) and P once. Scores of these inputs have
a standard deviation of at most 2.5, so key rounding moves a score by about
2.5 * 4e-4 = 1e-3 and a probability by 1e-3 of itself; values and P add 4e-4
and 2.8e-4: together 1.2e-3 rms, held to four times that, 5e-3 (rows are
averages over many keys, so the largest row error stays near the rms). bf16
outputs add 2^-8 of the value.
"""
import ctypes

import pytest
import torch

ADDR = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def kvq():
    import os
    from quantized_sparse_kv_gb300 import build, kvq as k
    if not os.path.exists(k.LIB_PATH):
        build.build()
    k.load_library()
    return k


def cache_struct(k, n=256, d=128, recent=128, kwin=1, hkv=2, b=1, vwin=1):
    return k.KvqCacheStruct(b, hkv, n, d, recent, kwin, vwin, ADDR, ADDR, ADDR, ADDR, ADDR, ADDR,
                            ADDR, (ctypes.c_uint32 * 4)(0, 0, 0, 0), 0, 0)


def test_refusals(kvq):
    lib = kvq.load_library()
    sz = ctypes.c_size_t(0)

    def call(c=None, q_dt=1, hq=16, t=8, t_dt=1, out_dt=1, q=ADDR, kt=ADDR, par=ADDR, ws=None,
             size=sz):
        c = c or cache_struct(kvq)
        return lib.kv_attend_tree(ctypes.byref(c), q, q_dt, hq, t, kt, ADDR, t_dt, par, 0.0, ADDR,
                                  out_dt, ws, ctypes.byref(size) if size is not None else None,
                                  None, None)
    assert call() == 0 and sz.value > 0                       # tensor path: partials
    assert call(q_dt=0) == 0 and sz.value == 0                # fp32 queries: no workspace
    assert call(t=256) == 0
    for kw in (dict(t=0), dict(t=257), dict(t=-1), dict(hq=3), dict(hq=0), dict(q_dt=2),
               dict(t_dt=2), dict(out_dt=2), dict(size=None)):
        assert call(**kw) == 1, kw
    big = ctypes.c_size_t(1 << 40)
    for kw in (dict(q=None), dict(kt=None), dict(par=None)):
        assert call(ws=ADDR, size=big, **kw) == 1, kw
    off = ctypes.c_void_p((1 << 20) + 4)
    for kw in (dict(q=off), dict(kt=off), dict(par=off), dict(ws=off)):
        assert call(**{**dict(ws=ADDR, size=big), **kw}) == 2, kw
    assert call(ws=ADDR, size=ctypes.c_size_t(16)) == 4
    assert call(c=cache_struct(kvq, hkv=1), q_dt=0, hq=65536) == 3
    bad = cache_struct(kvq)
    bad.k_codes = None
    assert call(c=bad) == 1


# ------------------------------------------------------------------ GPU
TOL_TENSOR, TOL_F32 = 5e-3, 1e-5


def make(kvq, b, hkv, n, d, recent, kwin="bf16", vwin="bf16", reserve=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if kwin == "f32" else torch.bfloat16
    k = torch.randn((b, hkv, n, d), generator=g, device="cuda").to(dt)
    v = torch.randn((b, hkv, n, d), generator=g, device="cuda").to(dt)
    return kvq.pack(k, v, recent, kwin, vwin, reserve=reserve)


def dequant(c, kvq):
    """Keys and values of the cache as attention reads them, fp64 (b, h, N, D)."""
    u = c.used()

    def codes(x):
        x = x.to(torch.int16)
        return torch.stack(((x & 15) - 8, (x >> 4) - 8), -1).flatten(-2).double()
    k = (codes(u["k_codes"]) * u["k_scales"].double().unsqueeze(3)).flatten(2, 3)[:, :, :c.cut]
    v = codes(u["v_codes"]) * u["v_scales"].double().repeat_interleave(32, -1)
    kw = u["k_window"]
    if c.kwin == kvq.MXFP8:
        e = c.k_window_e8m0[:, :, :c.recent].double().repeat_interleave(32, -1)
        kw = kw.contiguous().view(torch.float8_e4m3fn).double() * torch.exp2(e - 127)
    return torch.cat((k, kw.double()), 2), torch.cat((v, u["v_window"].double()), 2)


def ancestors(par):
    p = par.cpu().tolist()
    seen = torch.zeros((len(p), len(p[0]), len(p[0])), dtype=torch.bool)
    for b, row in enumerate(p):
        for i, x in enumerate(row):
            if x >= -1:
                seen[b, i, i] = True
            if x >= 0:
                seen[b, i] |= seen[b, x]
    return seen.to(par.device)


def plain(c, kvq, q, kt, vt, par):
    k, v = dequant(c, kvq)
    b, hq, t, d = q.shape
    g = hq // c.kv_heads
    seen = ancestors(par)
    out = torch.empty((b, hq, t, d), dtype=torch.float64, device=q.device)
    qq = q.double()
    if c.kwin == kvq.MXFP8:
        qq = mx_round(qq)
    for x in range(b):
        for h in range(hq):
            kk = torch.cat((k[x, h // g], kt[x, h // g].double()))
            vv = torch.cat((v[x, h // g], vt[x, h // g].double()))
            s = qq[x, h] @ kk.T / d ** 0.5
            s[:, c.n_tokens:] = torch.where(seen[x], s[:, c.n_tokens:], -torch.inf)
            p = torch.softmax(s, 1)
            live = p[:, c.n_tokens:] > 0
            # an unseen drafted row adds nothing, whatever it holds
            o = p[:, :c.n_tokens] @ vv[:c.n_tokens]
            for j in range(t):
                o = o + torch.where(live[:, j:j + 1], p[:, c.n_tokens + j, None] * vv[c.n_tokens + j], 0.0)
            out[x, h] = o
    return out


def mx_round(x):
    y = x.reshape(*x.shape[:-1], -1, 32)
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 8, torch.full_like(amax, -127.0))
    r = (y * torch.exp2(-e)).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    return (r * torch.exp2(e)).reshape(x.shape)


def random_tree(b, t, seed, pad=False):
    g = torch.Generator().manual_seed(seed)
    par = torch.empty((b, t), dtype=torch.int32)
    for x in range(b):
        for i in range(t):
            par[x, i] = int(torch.randint(-1, max(i, 0), (1,), generator=g)) if i else -1
        if pad and x % 2 == 0:
            n = int(torch.randint(0, t, (1,), generator=g))
            par[x, n:] = -2
    return par.cuda()


def inputs(b, hq, hkv, t, d, q_dt=torch.bfloat16, t_dt=torch.bfloat16, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (1.5 * torch.randn((b, hq, t, d), generator=g, device="cuda")).to(q_dt)
    k = torch.randn((b, hkv, t, d), generator=g, device="cuda").to(t_dt)
    v = torch.randn((b, hkv, t, d), generator=g, device="cuda").to(t_dt)
    return q, k, v


def compare(out, want, par, tol):
    live = (par > -2)[:, None, :, None].expand_as(out)
    err = torch.where(live, out.double() - want, 0.0)
    ref = torch.where(live, want, 0.0)
    if not bool(live.any()):
        return
    rel = float(err.norm() / ref.norm())
    assert rel <= tol, rel
    rows = err.norm(dim=-1) / ref.norm(dim=-1).clamp_min(1e-30)
    assert float(rows.max()) <= 4 * tol, float(rows.max())


CASES = [
    # b, hkv, G, n, recent, T
    (1, 1, 8, 128, 0, 1), (1, 2, 8, 1024, 128, 1), (2, 2, 8, 513, 130, 3),
    (1, 1, 1, 1, 1, 1), (1, 1, 1, 1, 0, 1), (2, 1, 8, 31, 7, 2), (3, 2, 8, 4100, 100, 16),
    (2, 2, 8, 1000, 128, 17), (1, 2, 8, 2048, 128, 33), (4, 2, 8, 700, 0, 64),
    (2, 1, 7, 333, 45, 19), (1, 3, 5, 900, 257, 50), (2, 1, 8, 200, 64, 128),
    (1, 1, 8, 300, 31, 256), (1, 4, 1, 640, 129, 130), (1, 1, 16, 8000, 128, 40),
    (33, 2, 8, 160, 32, 5), (1, 1, 12, 129, 129, 11),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("reserve", [False, True])
def test_tensor_path(kvq, case, reserve):
    b, hkv, g, n, recent, t = case
    gk = -(-(n - recent) // 32)
    c = make(kvq, b, hkv, n, 128, recent, reserve=(gk + 3, recent + 9) if reserve else None)
    q, k, v = inputs(b, g * hkv, hkv, t, 128)
    par = random_tree(b, t, n + t, pad=reserve)
    out = torch.full(q.shape, 7.0, device="cuda")
    call = kvq.AttendTree(c, q, k, v, par, out=out)
    call.run()
    assert kvq.read_status(call.status) == 0 and call.path == "tree_tensor"
    want = plain(c, kvq, q, k, v, par)
    compare(out, want, par, TOL_TENSOR)
    dead = (par == -2)[:, None, :, None].expand_as(out)
    assert bool((out[dead] == 7.0).all())  # rows without a token stay as they were
    first = out.clone()
    out.fill_(7.0)
    call.run()
    assert torch.equal(out, first)  # the same every time
    call16 = kvq.AttendTree(c, q, k, v, par)
    o16 = call16.run()
    assert kvq.read_status(call16.status) == 0
    err = (o16.double() - torch.where(dead, torch.zeros_like(first), first).double()).abs()
    assert bool((err <= 2.0 ** -8 * first.double().abs() + 1e-12).all() if not bool(dead.any())
                else (err[~dead] <= 2.0 ** -8 * first.double().abs()[~dead] + 1e-12).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d,kwin,vwin,q_dt,t_dt", [
    (128, "f32", "f32", torch.float32, torch.float32), (64, "bf16", "bf16", torch.bfloat16, torch.bfloat16),
    (32, "f32", "f32", torch.float32, torch.bfloat16), (256, "bf16", "f32", torch.float32, torch.float32),
    (96, "f32", "f32", torch.bfloat16, torch.float32), (128, "mxfp8", "bf16", torch.bfloat16, torch.bfloat16),
    (160, "bf16", "bf16", torch.float32, torch.bfloat16), (224, "f32", "f32", torch.float32, torch.float32),
])
def test_fp32_path(kvq, d, kwin, vwin, q_dt, t_dt):
    for b, hkv, g, n, recent, t in ((1, 1, 1, 1, 1, 1), (2, 2, 3, 150, 40, 7), (1, 1, 4, 97, 0, 35),
                                    (1, 2, 2, 70, 70, 65)):
        c = make(kvq, b, hkv, n, d, recent, kwin, vwin)
        q, k, v = inputs(b, g * hkv, hkv, t, d, q_dt, t_dt)
        par = random_tree(b, t, 3 * n, pad=True)
        out = torch.full(q.shape, 7.0, device="cuda")
        call = kvq.AttendTree(c, q, k, v, par, out=out)
        call.run()
        assert kvq.read_status(call.status) == 0 and call.path == "tree_rows"
        compare(out, plain(c, kvq, q, k, v, par), par, TOL_F32)
        assert bool((out[(par == -2)[:, None, :, None].expand_as(out)] == 7.0).all())


@pytest.mark.gpu
def test_chain_is_causal_and_agrees_with_the_appended_cache(kvq):
    # T new tokens under a chain: token i sees the cache and the new tokens up to i, which is
    # what kv_attend sees once tokens 0..i are in the cache's bf16 window
    b, hkv, n, t = 2, 2, 800, 6
    c = make(kvq, b, hkv, n, 128, 128, reserve=(40, 256))
    q, k, v = inputs(b, 16, hkv, t, 128)
    par = torch.arange(-1, t - 1, dtype=torch.int32, device="cuda").expand(b, t)
    out, st = kvq.attend_tree(c, q, k, v, par, out_dtype="f32")
    assert kvq.read_status(st) == 0
    for i in range(t):
        kvq.append(c, k[:, :, i:i + 1], v[:, :, i:i + 1], 128 + t)
        o, _, _ = kvq.attend(c, q[:, :, i:i + 1], out_dtype="f32")
        rel = float((o - out[:, :, i:i + 1]).norm() / o.norm())
        assert rel <= 2 * TOL_TENSOR, (i, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("q_dt", [torch.bfloat16, torch.float32])
def test_unseen_rows_never_reach_an_output(kvq, q_dt):
    b, hkv, n, t = 2, 1, 300, 24
    c = make(kvq, b, hkv, n, 128, 60)
    q, k, v = inputs(b, 8, hkv, t, 128, q_dt)
    par = random_tree(b, t, 9)
    par[:, 20:] = -2
    seen = ancestors(par)
    want = plain(c, kvq, q, k, v, par)
    bad = 3  # a drafted token with NaN and infinities, and everything behind the trees
    k[:, :, bad, ::2] = torch.nan
    v[:, :, bad, 0::3] = torch.inf
    v[:, :, bad, 1::3] = torch.nan
    for x in (q, k, v):
        x[:, :, 20:] = torch.nan
    out, st = kvq.attend_tree(c, q, k, v, par, out_dtype="f32")
    assert kvq.read_status(st) == 0
    free = ~seen[:, :, bad] & (par > -2)
    rows = free[:, None, :, None].expand_as(out)
    assert bool(rows.any()) and bool(torch.isfinite(out[rows]).all())
    tol = TOL_TENSOR if q_dt == torch.bfloat16 else TOL_F32
    err = torch.where(rows, out.double() - want, 0.0).norm()
    assert float(err / torch.where(rows, want, 0.0).norm()) <= tol
    hit = (seen[:, :, bad] & (par > -2))[:, None, :, None].expand_as(out)
    assert not bool(torch.isfinite(out[hit]).any())
    # an infinity in V alone reaches exactly the rows that see it, and only its features
    k2, v2 = torch.randn_like(k), torch.randn_like(v)
    q2 = torch.randn_like(q)
    v2[:, :, bad, 5] = torch.inf
    out, _ = kvq.attend_tree(c, q2, k2, v2, par, out_dtype="f32")
    assert bool((out[..., 5][(seen[:, :, bad] & (par > -2))[:, None].expand_as(out[..., 5])]
                 == torch.inf).all())
    ok = torch.isfinite(out) | (par == -2)[:, None, :, None]
    ok[..., 5] |= seen[:, :, bad][:, None]
    assert bool(ok.all())


@pytest.mark.gpu
@pytest.mark.parametrize("q_dt", [torch.bfloat16, torch.float32])
def test_bad_parents_are_flagged_and_left_out(kvq, q_dt):
    b, hkv, n, t = 1, 2, 260, 10
    c = make(kvq, b, hkv, n, 128, 33)
    q, k, v = inputs(b, 16, hkv, t, 128, q_dt)
    good = torch.tensor([[-1, 0, 1, -1, 3, -2, 0, 6, 2, -1]], dtype=torch.int32, device="cuda")
    for i, value in ((4, 4), (4, 9), (4, 1 << 30), (4, -3), (4, -(1 << 31)), (6, 5)):
        par = good.clone()
        par[0, i] = value
        ref = good.clone()  # the row and those behind it hold no token
        ref[0, i] = -2
        if i == 6:
            ref[0, 7] = -2
        out = torch.full(q.shape, 7.0, device="cuda")
        call = kvq.AttendTree(c, q, k, v, par, out=out)
        call.run()
        assert kvq.read_status(call.status) == kvq.DEV_INDEX, (i, value)
        want = torch.full(q.shape, 7.0, device="cuda")
        ok = kvq.AttendTree(c, q, k, v, ref, out=want)
        ok.run()
        assert kvq.read_status(ok.status) == 0
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_large_scores_and_flat_ones(kvq):
    # scores that grow along the cache (the reference is raised again and again), and equal ones
    b, hkv, n, t, d = 1, 1, 3000, 9, 128
    ramp = torch.linspace(0.02, 6.0, n, device="cuda")[None, None, :, None]
    base = torch.randn((1, 1, 1, d), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    k = (ramp * base).bfloat16()
    v = torch.randn((b, hkv, n, d), device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    c = kvq.pack(k, v, 128, "bf16")
    q, kt, vt = inputs(b, 8, hkv, t, d)
    q = (q * 0 + 2 * base.sign() + 0.1 * q).bfloat16()
    par = random_tree(b, t, 4)
    out, st = kvq.attend_tree(c, q, kt, vt, par, out_dtype="f32")
    assert kvq.read_status(st) == 0
    # scores reach 6 * 2 * 128 * 0.8 / 11.3 = 110: rounding a key by 4e-4 moves one by 110 * 4e-4
    # / sqrt(128) * 1.25 = 5e-3 and the row's few leading probabilities by as much
    compare(out, plain(c, kvq, q, kt, vt, par), par, 2e-2)
    zero = torch.zeros_like(q)
    out, _ = kvq.attend_tree(c, zero, kt, vt, par, out_dtype="f32")
    compare(out, plain(c, kvq, zero, kt, vt, par), par, TOL_TENSOR)


@pytest.mark.gpu
def test_graphs_streams_and_growing_cache(kvq):
    b, hkv, n, t = 2, 2, 896, 8
    c = make(kvq, b, hkv, n, 128, 128, reserve=(200, 512))
    q, k, v = inputs(b, 16, hkv, t, 128)
    par = random_tree(b, t, 6)
    a1, a2 = kvq.AttendTree(c, q, k, v, par), kvq.AttendTree(c, -q, k, v, par)
    w1, w2 = a1.run().clone(), a2.run().clone()
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a in (a1, a2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a.run()
        graphs.append(g)
    a1.out.zero_()
    a2.out.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, g in zip(streams, graphs):  # two calls at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a1.out, w1) and torch.equal(a2.out, w2)
    # a prepared call follows the cache as it grows, workspace included
    for _ in range(3):
        x = torch.randn((b, hkv, 700, 128), device="cuda").bfloat16()
        for i in range(0, 700, 100):
            kvq.append(c, x[:, :, i:i + 100], x[:, :, i:i + 100], 128)
        a1.run()
        assert kvq.read_status(a1.status) == 0
        compare(a1.out, plain(c, kvq, q, k, v, par), par, TOL_TENSOR + 2.0 ** -8)


@pytest.mark.gpu
def test_wait_that_runs_out_is_reported(kvq):
    # a key tile that never arrives: the call ends with KVQ_DEV_TIMEOUT after a short limit, the
    # next one is right again
    b, hkv, n, t = 1, 2, 5000, 8
    c = make(kvq, b, hkv, n, 128, 128)
    q, k, v = inputs(b, 16, hkv, t, 128)
    par = random_tree(b, t, 6)
    call = kvq.AttendTree(c, q, k, v, par)
    want = call.run().clone()
    assert kvq.read_status(call.status) == 0
    kvq.debug_set(wait_limit_ns=2_000_000, drop_item=5)
    try:
        call.run()
        torch.cuda.synchronize()
    finally:
        kvq.debug_set()
    assert kvq.read_status(call.status) == kvq.DEV_TIMEOUT
    call.status.zero_()
    assert torch.equal(call.run(), want)
    assert kvq.read_status(call.status) == 0


@pytest.mark.gpu
def test_outgrown_workspace_is_kept_for_captured_graphs(kvq):
    """A graph captured before the cache grew writes to the workspace of that time."""
    import weakref
    b, hq, hkv, t = 2, 16, 2, 8
    c = make(kvq, b, hkv, 256, 128, 128, reserve=(600, 512))
    q, kt, vt = inputs(b, hq, hkv, t, 128)
    par = random_tree(b, t, 3)
    calls = [kvq.AttendTree(c, q, kt, vt, par),
             kvq.AttendBlocks(c, q, kvq.BlockSummary(c, 32).update(), 512)]
    refs = [weakref.ref(a.ws) for a in calls]
    sizes = [a.ws.numel() for a in calls]
    new = torch.randn((b, hkv, 320, 128), device="cuda", dtype=torch.bfloat16)
    for _ in range(50):
        kvq.append(c, new, new, 128)
    calls[1].summary.update()
    for a in calls:
        a.run()
    torch.cuda.synchronize()
    for a, ref, size in zip(calls, refs, sizes):
        assert a.ws.numel() >= size * 3 // 2 and ref() is not None


@pytest.mark.gpu
def test_leaves_that_are_copied_record_nothing(kvq):
    """Inputs a call cannot read in place are copied again each run, without a
    gradient history that would grow with the runs."""
    b, hq, hkv, t = 1, 16, 2, 4
    c = make(kvq, b, hkv, 160, 128, 128)
    q, kt, vt = inputs(b, hq, hkv, t, 128)
    par = random_tree(b, t, 3)
    want = kvq.AttendTree(c, q, kt, vt, par).run()
    leaf = q.transpose(1, 2).contiguous().requires_grad_()
    a = kvq.AttendTree(c, leaf.transpose(1, 2), kt, vt, par)
    s = kvq.AttendBlocks(c, leaf.transpose(1, 2), kvq.BlockSummary(c, 32).update(), 1)
    wide = torch.zeros((b, 2, 64, 8), device="cuda", requires_grad=True)
    r = kvq.Rope(kvq.RopePlan(64), wide.transpose(2, 3), None,
                 torch.zeros((b, 8), device="cuda", dtype=torch.int64))
    for x in (a, s, r):
        x.run()
        assert len(x._copies) > 0 and not any(y.requires_grad for y, _ in x._copies)
    assert torch.equal(a.out, want)
    with torch.no_grad():
        leaf.mul_(0.0)  # the next run reads the leaf's new values
    assert not torch.equal(a.run(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(3, 2, 8, 4100, 100, 16), (1, 2, 8, 16384, 128, 33),
                                  (8, 2, 8, 6000, 112, 8)])
def test_many_runs_agree(kvq, case):
    """The hand-overs between the kernel's warps leave nothing to timing: each of many
    runs back to back gives the same bits (two tiles a block, and several)."""
    b, hkv, g, n, recent, t = case
    c = make(kvq, b, hkv, n, 128, recent)
    q, k, v = inputs(b, g * hkv, hkv, t, 128)
    par = random_tree(b, t, n + t)
    call = kvq.AttendTree(c, q, k, v, par, out_dtype="f32")
    first = call.run().clone()
    compare(first, plain(c, kvq, q, k, v, par), par, TOL_TENSOR)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        differ += (call.run() != first).any()
    assert int(differ) == 0 and kvq.read_status(call.status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,g", [(64, 1), (64, 3), (96, 6), (224, 5), (256, 9)])
def test_fp32_path_shared_heads(kvq, d, g):
    """Query heads share the fp32 kernel's keys four at a time: whole groups and parts."""
    b, hkv, t = 2, 2, 9
    c = make(kvq, b, hkv, 420, d, 37)
    q, k, v = inputs(b, g * hkv, hkv, t, d)
    par = random_tree(b, t, d + g, pad=True)
    out = torch.full(q.shape, 7.0, device="cuda")
    a = kvq.AttendTree(c, q, k, v, par, out=out)
    a.run()
    assert kvq.read_status(a.status) == 0 and a.path == "tree_rows"
    compare(out, plain(c, kvq, q, k, v, par), par, TOL_F32)
    dead = (par == -2)[:, None, :, None].expand_as(out)
    assert bool((out[dead] == 7.0).all())
