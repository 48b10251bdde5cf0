"""Block summaries, the choice of blocks and attention over chosen blocks.

Summaries and choices are defined by integers and single fp32 roundings, so the
GPU's are compared for equality with a plain form that rounds at the same
places. Attention over the chosen blocks: the fp32 kernel's relative L2 within
1e-5, the decode kernels' within 5e-3 (their q' = q * scale, values and
probabilities are rounded to fp16, 2^-11 each; see test_tree.py for how such
roundings reach an output).
"""
import ctypes

import numpy as np
import pytest
import torch

from test_tree import cache_struct, dequant, kvq, make, mx_round  # noqa: F401 (fixture)

ADDR = ctypes.c_void_p(1 << 20)
TOL_DECODE, TOL_F32 = 5e-3, 1e-5


def test_refusals(kvq):  # noqa: F811
    lib = kvq.load_library()
    c = cache_struct(kvq, n=1000, recent=100)   # 900 int4 tokens: 15 blocks of 64
    sz = ctypes.c_size_t(0)

    def summary(block=64, cap=15, codes=ADDR, scales=ADDR):
        return kvq.KvqSummary(codes, scales, block, cap)

    def build(s, first=99):
        return lib.kv_block_summary(ctypes.byref(c), ctypes.byref(s) if s else None, first, None,
                                    None)
    assert build(summary()) == 0 and lib.kvq_last_launch_count() == 0   # nothing past the last
    assert build(None) == 1
    assert build(summary(block=48)) == 1 and build(summary(block=256)) == 1
    assert build(summary(cap=14)) == 4
    assert build(summary(codes=None)) == 1 and build(summary(scales=None)) == 1
    assert build(summary(codes=ctypes.c_void_p((1 << 20) + 8))) == 2
    assert build(summary(), first=-1) == 1

    def values(s, first=0, out=ADDR):
        return lib.kv_block_values(ctypes.byref(c), ctypes.byref(s) if s else None, first, out,
                                   None, None)
    assert values(summary(), first=15, out=None) == 0 and lib.kvq_last_launch_count() == 0
    assert values(None) == 1 and values(summary(), first=-1) == 1
    assert values(summary(), out=None) == 1
    assert values(summary(), out=ctypes.c_void_p((1 << 20) + 4)) == 2

    def select(cc=c, hq=16, nq=1, top=4, sink=1, dt=1, ws=None, size=sz, sel=ADDR, q=ADDR):
        return lib.kv_select_blocks(ctypes.byref(cc), ctypes.byref(summary()), q, dt, hq, nq, top,
                                    sink, sel, ws, ctypes.byref(size) if size is not None else None,
                                    None, None)
    assert select() == 0 and sz.value == 4 * 2 * 16        # score rows padded to four
    assert select(top=15) == 0 and sz.value == 0          # every block: nothing to score
    for kw in (dict(top=0), dict(sink=-1), dict(sink=5), dict(hq=3), dict(nq=0), dict(dt=2),
               dict(size=None)):
        assert select(**kw) == 1, kw
    big = ctypes.c_size_t(1 << 30)
    assert select(ws=ADDR, size=big, sel=None) == 1 and select(ws=ADDR, size=big, q=None) == 1
    assert select(ws=ADDR, size=ctypes.c_size_t(8)) == 4
    assert select(ws=ADDR, size=big, q=ctypes.c_void_p((1 << 20) + 2)) == 2
    assert select(hq=130) == 3 and select(nq=32768) == 3

    def attend(hq=16, nq=1, top=4, block=64, dt=1, out=1, ws=None, size=sz, sel=ADDR):
        return lib.kv_attend_blocks(ctypes.byref(c), ADDR, dt, hq, nq, sel, top, block, 0.0, ADDR,
                                    out, ws, ctypes.byref(size) if size is not None else None, None,
                                    None)
    assert attend() == 0 and sz.value > 0
    assert attend(dt=0) == 0 and sz.value == 0            # fp32 queries: the fp32 kernel
    for kw in (dict(top=0), dict(block=16), dict(hq=3), dict(nq=0), dict(dt=2), dict(out=2),
               dict(size=None)):
        assert attend(**kw) == 1, kw
    assert attend(ws=ADDR, size=big, sel=None) == 1
    assert attend(ws=ADDR, size=ctypes.c_size_t(8)) == 4
    assert attend(hq=131072, dt=0) == 3
    assert attend(top=0x7fffffff, dt=0) == 0 and attend(top=0x7fffffff) == 0


def test_binding_refusals(kvq):  # noqa: F811
    class Fake:
        n_tokens = 0
    with pytest.raises(ValueError):
        kvq.BlockSummary(Fake(), 48)


# ------------------------------------------------------------------ GPU


def plain_summary(c, block):
    """Codes and scales by the definition, numpy fp32."""
    u = c.used()
    kc = u["k_codes"].cpu().numpy().astype(np.int32)
    codes = np.stack(((kc & 15) - 8, (kc >> 4) - 8), -1).reshape(*kc.shape[:-1], 2 * kc.shape[-1])
    part = u["k_scales"].cpu().numpy() * codes.sum(3).astype(np.float32)
    b, h, gk, d = part.shape
    m, blocks = block // 32, -(-c.cut // block)
    mean = np.zeros((b, h, blocks, d), np.float32)
    for j in range(blocks):
        acc = part[:, :, j * m]
        for g in range(j * m + 1, min(gk, (j + 1) * m)):
            acc = acc + part[:, :, g]
        mean[:, :, j] = acc / np.float32(min(block, c.cut - j * block))
    scale = np.abs(mean).max(-1, initial=0) / np.float32(127)
    safe = np.where(scale > 0, scale, np.float32(1))[..., None]
    return np.where(scale[..., None] > 0, np.rint(mean / safe), 0).astype(np.int8), scale


def plain_select(q, codes, scales, hkv, top_k, sink):
    q = q.float().cpu().numpy()
    b, hq, nq, d = q.shape
    g, blocks = hq // hkv, codes.shape[2]
    out = np.full((b, hkv, nq, top_k), -1, np.int32)
    sq = np.abs(q).max(-1) / np.float32(127)
    qi = np.where(sq[..., None] > 0, np.rint(q / np.where(sq > 0, sq, np.float32(1))[..., None]), 0)
    for x in range(b):
        for h in range(hkv):
            for i in range(nq):
                best = np.full(blocks, -np.inf, np.float32)
                for j in range(h * g, (h + 1) * g):
                    dot = (codes[x, h].astype(np.int64) @ qi[x, j, i].astype(np.int64)).astype(np.float32)
                    best = np.maximum(best, (sq[x, j, i] * scales[x, h]) * dot)
                best[:sink] = np.inf
                best = best + np.float32(0)
                order = np.lexsort((np.arange(blocks), -best))[:top_k]
                out[x, h, i, :len(order)] = np.sort(order)
    return out


def plain_attend(c, kvq, q, sel, block):  # noqa: F811
    k, v = dequant(c, kvq)
    b, hq, nq, d = q.shape
    g = hq // c.kv_heads
    qq = mx_round(q.double()) if c.kwin == kvq.MXFP8 else q.double()
    out = torch.zeros((b, hq, nq, d), dtype=torch.float64, device=q.device)
    lists = sel.cpu().tolist()
    for x in range(b):
        for h in range(hq):
            for i in range(nq):
                see = torch.zeros(c.n_tokens, dtype=torch.bool, device=q.device)
                see[c.cut:] = True
                for e in lists[x][h // g][i]:
                    if e >= 0:
                        see[e * block:min((e + 1) * block, c.cut)] = True
                if not bool(see.any()):
                    continue
                s = k[x, h // g][see] @ qq[x, h, i] / d ** 0.5
                out[x, h, i] = torch.softmax(s, 0) @ v[x, h // g][see]
    return out


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def query(b, hq, nq, d, dt=torch.bfloat16, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1.5 * torch.randn((b, hq, nq, d), generator=g, device="cuda")).to(dt)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 224, 256])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_summary(kvq, d, block):  # noqa: F811
    for b, h, n, recent, reserve in ((1, 1, 1, 0, False), (2, 2, 300, 40, True), (1, 3, 129, 1, False),
                                     (3, 1, 700, 60, True), (1, 1, 33, 33, True)):
        gk = -(-(n - recent) // 32)
        c = make(kvq, b, h, n, d, recent, "f32", "f32", reserve=(gk + 5, recent + 3) if reserve else None)
        s = kvq.BlockSummary(c, block)
        s.codes.fill_(99)
        s.scales.fill_(99.0)
        s.update()
        codes, scales = plain_summary(c, block)
        nb = s.blocks
        assert np.array_equal(s.codes[:, :, :nb].cpu().numpy(), codes)
        assert np.array_equal(s.scales[:, :, :nb].cpu().numpy(), scales)
        assert bool((s.codes[:, :, nb:] == 99).all()) and bool((s.scales[:, :, nb:] == 99).all())
        if nb > 1:  # from a later block on: the ones before stay
            s.codes.fill_(99)
            s.update(first=nb - 1)
            assert bool((s.codes[:, :, :nb - 1] == 99).all())
            assert np.array_equal(s.codes[:, :, nb - 1:nb].cpu().numpy(), codes[:, :, nb - 1:])
        v = s.update().values()
        assert v.shape == (b, h, nb, d)
        assert torch.equal(v.cpu(), torch.from_numpy(codes.astype(np.float32) * scales[..., None]))


@pytest.mark.gpu
def test_summary_of_zero_keys(kvq):  # noqa: F811
    z = torch.zeros((1, 1, 256, 128), device="cuda").bfloat16()
    c = kvq.pack(z, z, 0, "bf16")
    s = kvq.BlockSummary(c, 64).update()
    assert not bool(s.codes.any()) and not bool(s.scales.any())
    out, sel, st = kvq.attend_blocks(c, query(1, 8, 1, 128), s, 2)
    assert sel.cpu().tolist() == [[[[0, 1]]]] and kvq.read_status(st) == 0  # all equal: the lowest
    assert not bool(out.any())


SELECT = [
    # b, hkv, G, nq, n, recent, d, block, top_k, sink, q type
    (2, 2, 8, 1, 5000, 128, 128, 32, 7, 1, torch.bfloat16),
    (1, 1, 8, 3, 9000, 100, 128, 32, 200, 0, torch.bfloat16),
    (1, 2, 1, 1, 700, 0, 128, 64, 1, 0, torch.float32),
    (2, 1, 7, 2, 1111, 55, 64, 32, 13, 2, torch.bfloat16),
    (1, 1, 12, 1, 2000, 32, 256, 128, 5, 5, torch.float32),
    (1, 1, 64, 1, 900, 4, 32, 32, 9, 0, torch.bfloat16),
    (1, 2, 8, 1, 300, 44, 128, 64, 64, 1, torch.bfloat16),    # fewer blocks than top_k
    (1, 2, 8, 1, 60, 60, 128, 64, 3, 1, torch.bfloat16),      # no block at all
    (1, 1, 8, 1, 40000, 0, 96, 32, 256, 3, torch.bfloat16),
    (1, 1, 8, 2, 40000, 0, 128, 32, 100, 1, torch.bfloat16),   # one piece of keys
    (1, 2, 4, 1, 131072, 60, 128, 32, 33, 0, torch.bfloat16),
    (1, 1, 8, 1, 400000, 0, 128, 32, 64, 2, torch.bfloat16),   # several pieces
    (1, 1, 2, 1, 600000, 0, 128, 32, 40, 1, torch.bfloat16),
    (1, 1, 9, 1, 8195, 3, 128, 64, 31, 0, torch.bfloat16),
    (2, 1, 8, 1, 32 * 256, 0, 128, 32, 255, 0, torch.float32),
    (2, 1, 8, 1, 32 * 257, 0, 128, 32, 256, 0, torch.float32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SELECT)
def test_select(kvq, case):  # noqa: F811
    b, h, g, nq, n, recent, d, block, top, sink, dt = case
    c = make(kvq, b, h, n, d, recent, reserve=(-(-(n - recent) // 32) + 2, recent + 1))
    s = kvq.BlockSummary(c, block).update()
    q = query(b, g * h, nq, d, dt)
    a = kvq.AttendBlocks(c, q, s, top, n_sink=sink)
    a.selected.fill_(77)
    a.run()
    assert kvq.read_status(a.status) == 0
    codes, scales = plain_summary(c, block)
    want = plain_select(q, codes, scales, h, top, sink)
    assert np.array_equal(a.selected.cpu().numpy(), want)


@pytest.mark.gpu
def test_select_ties_go_to_the_lower_block(kvq):  # noqa: F811
    # keys repeat every 64 tokens within runs of blocks: many equal scores around the border
    one = torch.randn((1, 1, 64, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    gain = torch.tensor([1.0, 2.0, 1.0, 1.0, 0.5, 2.0, 1.0, 1.0] * 8, device="cuda")
    k = (one.unsqueeze(2) * gain[None, None, :, None, None]).flatten(2, 3).bfloat16()
    c = kvq.pack(k, k, 0, "bf16")
    s = kvq.BlockSummary(c, 64).update()
    q = query(1, 8, 1, 128)
    codes, scales = plain_summary(c, 64)
    for top in (1, 3, 15, 16, 17, 18, 40, 55, 57, 63):
        for sink in (0, 1):
            a = kvq.AttendBlocks(c, q, s, top, n_sink=sink)
            a.run()
            assert np.array_equal(a.selected.cpu().numpy(), plain_select(q, codes, scales, 1, top, sink))


ATTEND = [
    # b, hkv, G, nq, n, recent, block, top_k
    (1, 2, 8, 1, 4000, 128, 64, 8), (2, 1, 8, 3, 1500, 100, 32, 11), (1, 2, 4, 1, 900, 0, 64, 3),
    (2, 1, 7, 2, 777, 77, 128, 2), (1, 1, 1, 1, 500, 9, 32, 6), (1, 1, 8, 1, 129, 0, 128, 4),
    (1, 2, 8, 1, 90, 90, 64, 2), (40, 2, 8, 1, 700, 64, 32, 5), (1, 1, 8, 1, 20000, 130, 32, 400),
    (1, 1, 8, 70, 600, 33, 64, 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTEND)
def test_attend_decode_kernels(kvq, case):  # noqa: F811
    b, h, g, nq, n, recent, block, top = case
    c = make(kvq, b, h, n, 128, recent, reserve=(-(-(n - recent) // 32) + 2, recent + 1))
    s = kvq.BlockSummary(c, block).update()
    q = query(b, g * h, nq, 128)
    a = kvq.AttendBlocks(c, q, s, top, out_dtype="f32")
    out = a.run()
    assert kvq.read_status(a.status) == 0 and a.path == "blocks_decode"
    assert rel(out, plain_attend(c, kvq, q, a.selected, block)) <= TOL_DECODE
    o16 = kvq.AttendBlocks(c, q, s, top).run()
    assert bool(((o16.double() - out.double()).abs() <= 2.0 ** -8 * out.double().abs() + 1e-12).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d,kwin,vwin,dt,g", [
    (128, "f32", "f32", torch.float32, 8), (64, "bf16", "bf16", torch.bfloat16, 4),
    (32, "f32", "f32", torch.bfloat16, 3), (256, "bf16", "f32", torch.float32, 2),
    (128, "bf16", "bf16", torch.bfloat16, 16), (128, "mxfp8", "bf16", torch.bfloat16, 8),
    (96, "f32", "bf16", torch.float32, 1)])
def test_attend_fp32_kernel(kvq, d, kwin, vwin, dt, g):  # noqa: F811
    for b, h, nq, n, recent, block, top in ((1, 2, 2, 700, 50, 32, 5), (2, 1, 1, 300, 0, 64, 3),
                                            (1, 1, 1, 45, 45, 32, 2)):
        c = make(kvq, b, h, n, d, recent, kwin, vwin)
        s = kvq.BlockSummary(c, block).update()
        q = query(b, g * h, nq, d, dt)
        a = kvq.AttendBlocks(c, q, s, top, out_dtype="f32")
        out = a.run()
        assert kvq.read_status(a.status) == 0 and a.path == "blocks_rows"
        assert rel(out, plain_attend(c, kvq, q, a.selected, block)) <= TOL_F32


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_lists_of_the_caller(kvq, dt):  # noqa: F811
    b, h, nq, n, recent, block = 1, 2, 1, 640, 0, 64       # 10 blocks, no window
    c = make(kvq, b, h, n, 128, recent)
    q = query(b, 16, nq, 128, dt)
    tol = TOL_DECODE if dt == torch.bfloat16 else TOL_F32

    def run(rows):
        sel = torch.tensor([[[r] for r in rows]], dtype=torch.int32, device="cuda")
        a = kvq.AttendBlocks(c, q, None, sel.shape[-1], out_dtype="f32", selected=sel, block=block)
        out = a.run(select=False)
        return out, kvq.read_status(a.status)

    def want(rows):
        sel = torch.tensor([[[r] for r in rows]], dtype=torch.int32)
        return plain_attend(c, kvq, q, sel, block)
    out, st = run([[0, 3, 9], [4, -1, -1]])
    assert st == 0 and rel(out, want([[0, 3, 9], [4, -1, -1]])) <= tol
    out, st = run([[-1, -1, -1], [2, 5, -1]])               # an empty row is zero
    assert st == 0 and not bool(out[:, :8].any())
    assert rel(out, want([[-1, -1, -1], [2, 5, -1]])) <= tol
    # entries outside the blocks are skipped and flagged
    for bad in (10, 1 << 30, -2, -(1 << 31)):
        out, st = run([[0, bad, -1], [4, 5, 6]])
        assert st == kvq.DEV_INDEX, bad
        assert rel(out, want([[0, -1, -1], [4, 5, 6]])) <= tol
    out, st = run([[0, -1, 3], [4, 5, 6]])                  # an entry behind the end
    assert st == kvq.DEV_INDEX
    assert rel(out, want([[0, -1, -1], [4, 5, 6]])) <= tol
    # entries past the tenth (as many as there are blocks) are not looked at
    long = list(range(10)) + [99, 3]
    out, st = run([long, long])
    assert st == 0 and rel(out, want([long[:10] + [-1, -1]] * 2)) <= tol
    # the same index twice, or a list that is not increasing
    for rows in ([[3, 3, -1], [4, 5, 6]], [[5, 3, -1], [4, 5, 6]]):
        _, st = run(rows)
        assert st == kvq.DEV_DUP


@pytest.mark.gpu
def test_all_blocks_is_dense_attention(kvq):  # noqa: F811
    c = make(kvq, 2, 2, 1300, 128, 128)
    q = query(2, 16, 1, 128)
    s = kvq.BlockSummary(c, 64).update()
    out, sel, st = kvq.attend_blocks(c, q, s, 40, out_dtype="f32")
    dense, _, path = kvq.attend(c, q, out_dtype="f32")
    assert kvq.read_status(st) == 0 and path == "decode"
    assert rel(out, dense.double()) <= 2 * TOL_DECODE


@pytest.mark.gpu
def test_captured_streams_and_wait(kvq):  # noqa: F811
    c = make(kvq, 2, 2, 3100, 128, 128)
    s = kvq.BlockSummary(c, 64).update()
    q = query(2, 16, 1, 128)
    a1, a2 = kvq.AttendBlocks(c, q, s, 9), kvq.AttendBlocks(c, -q, s, 9)
    w = [x.run().clone() for x in (a1, a2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a in (a1, a2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.update()
            a.run()
        graphs.append(g)
        a.out.zero_()
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a1.out, w[0]) and torch.equal(a2.out, w[1])
    kvq.debug_set(wait_limit_ns=2_000_000, drop_item=1)
    try:
        a1.run()
        torch.cuda.synchronize()
    finally:
        kvq.debug_set()
    assert kvq.read_status(a1.status) == kvq.DEV_TIMEOUT
    a1.status.zero_()
    assert torch.equal(a1.run(), w[0]) and kvq.read_status(a1.status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("g,nq,n,dt", [(12, 3, 3000, torch.bfloat16), (33, 1, 5000, torch.float32),
                                       (64, 2, 900, torch.bfloat16), (2, 5, 4100, torch.float32)])
def test_select_many_heads(kvq, g, nq, n, dt):  # noqa: F811
    """Head counts that fill eight columns of the scores' MMA several times, or in part."""
    c = make(kvq, 2, 1, n, 128, 36)
    s = kvq.BlockSummary(c, 32).update()
    q = query(2, g, nq, 128, dt)
    a = kvq.AttendBlocks(c, q, s, 9, n_sink=1)
    a.run()
    assert kvq.read_status(a.status) == 0
    codes, scales = plain_summary(c, 32)
    assert np.array_equal(a.selected.cpu().numpy(), plain_select(q, codes, scales, 1, 9, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("d,g", [(64, 1), (64, 3), (96, 6), (224, 5), (256, 9)])
def test_attend_fp32_kernel_shared_heads(kvq, d, g):  # noqa: F811
    """Query heads share the fp32 kernel's keys four at a time: whole groups and parts."""
    c = make(kvq, 2, 2, 500, d, 41)
    q = query(2, 2 * g, 2, d)
    a = kvq.AttendBlocks(c, q, kvq.BlockSummary(c, 64).update(), 3, out_dtype="f32")
    out = a.run()
    assert kvq.read_status(a.status) == 0 and a.path == "blocks_rows"
    assert rel(out, plain_attend(c, kvq, q, a.selected, 64)) <= TOL_F32


@pytest.mark.gpu
def test_out_decides_the_output_type(kvq):  # noqa: F811
    c = make(kvq, 1, 2, 300, 128, 44)
    q = query(1, 16, 1, 128)
    s = kvq.BlockSummary(c, 32).update()
    want = kvq.AttendBlocks(c, q, s, 4, out_dtype="f32").run()
    out = torch.empty(q.shape, device="cuda")
    assert kvq.AttendBlocks(c, q, s, 4, out=out).run() is out and torch.equal(out, want)
    with pytest.raises(ValueError):
        kvq.AttendBlocks(c, q, s, 4, out=out.half())
