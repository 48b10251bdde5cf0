"""The calls of a decoding step in a row, as a serving loop makes them.

A speculative step: rotary positions of the drafted tokens' queries and keys at
their depths, attention of the tree over the cache, the accepted path appended to
the cache; then a block-sparse step on the grown cache: summaries of the new
blocks, the choice of blocks, attention over them. Every output is compared with
a 64-bit computation that keeps its own copy of the sequence, and the grown cache
with kv_pack of the whole sequence. Tolerances as in test_tree.py (fp16 operands,
5e-3 relative L2); rotated bf16 rows add 2^-8 of an element, which both sides see,
since the comparison takes the library's rotated rows (checked for themselves).
"""
import pytest
import torch

from test_blocks import plain_attend, plain_select, plain_summary
from test_tree import TOL_TENSOR, ancestors, compare, dequant, kvq, plain  # noqa: F401 (fixture)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,n,window", [(2, 640, 64), (3, 1376, 128)])
def test_speculative_then_sparse_steps(kvq, batch, n, window):  # noqa: F811
    hq, hkv, d, block, top = 16, 2, 128, 64, 6
    gen = torch.Generator(device="cuda").manual_seed(n)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    plan = kvq.RopePlan(d, scaling="bands", factor=4.0, original=4096, low=1.0, high=4.0)
    pos0 = torch.arange(n, device="cuda", dtype=torch.int32).expand(batch, n)
    keys = kvq.rope(plan, rand(batch, hkv, n, d), None, pos0)[0]
    values = rand(batch, hkv, n, d)
    cache = kvq.pack(keys, values, window, "bf16", reserve=(n // 32 + 20, window + 64))
    summary = kvq.BlockSummary(cache, block).update()
    plan_freq = [t / 2.0 ** 64 * 6.283185307179586 for t in plan.turns_host]
    for step in range(4):
        # ---- a drafted tree of 7 tokens, two branches behind its root
        par = torch.tensor([[-1, 0, 0, 1, 2, 3, 4]], dtype=torch.int32, device="cuda")
        par = par.expand(batch, 7).contiguous()
        depth = torch.tensor([0, 1, 1, 2, 2, 3, 3], dtype=torch.int32, device="cuda")
        rows = rand(batch, 7, hq + 2 * hkv, d)  # the projection's rows of the drafted tokens
        q, k, v = (rows[:, :, i:j].transpose(1, 2) for i, j in
                   ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        pos = (cache.n_tokens + depth).expand(batch, 7)
        rq, rk, rv = kvq.rope(plan, q, k, pos, v=v)
        ang = pos.double()[:, None, :, None] * torch.tensor(plan_freq, dtype=torch.float64,
                                                            device="cuda")
        a, b = q.double()[..., :64], q.double()[..., 64:]
        want = torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)
        assert bool(((rq.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2e-5).all())
        assert torch.equal(rv, v)
        call = kvq.AttendTree(cache, rq, rk, rv, par, out_dtype="f32")
        out = call.run()
        assert kvq.read_status(call.status) == 0
        compare(out, plain(cache, kvq, rq, rk, rv, par), par, TOL_TENSOR)
        # ---- the branch 0, 2, 4 is accepted
        take = [0, 2, 4]
        old_cut = cache.cut
        kvq.append(cache, rk[:, :, take], rv[:, :, take], window)
        keys = torch.cat((keys, rk[:, :, take]), 2)
        values = torch.cat((values, rv[:, :, take]), 2)
        assert cache.n_tokens == keys.shape[2]
        summary.update(first=old_cut // block)
        whole = kvq.pack(keys, values, cache.recent, "bf16")
        for name, view in cache.used().items():
            assert torch.equal(view, whole.used()[name]), name
        codes, scales = plain_summary(cache, block)
        assert (summary.codes[:, :, :summary.blocks].cpu().numpy() == codes).all()
        # ---- a block-sparse step of the next token
        q1 = rand(batch, hq, 1, d)
        p1 = torch.full((batch, 1), cache.n_tokens, device="cuda")
        q1 = kvq.rope(plan, q1, None, p1)[0]
        o, sel, st = kvq.attend_blocks(cache, q1, summary, top, n_sink=1, out_dtype="f32")
        assert kvq.read_status(st) == 0
        assert (sel.cpu().numpy() == plain_select(q1, codes, scales, hkv, top, 1)).all()
        want = plain_attend(cache, kvq, q1, sel, block)
        assert float((o.double() - want).norm() / want.norm()) <= TOL_TENSOR
        # many more tokens, so that groups migrate and blocks complete
        more = 45
        ks, vs = rand(batch, hkv, more, d), rand(batch, hkv, more, d)
        old_cut = cache.cut
        kvq.append(cache, ks, vs, window)
        keys, values = torch.cat((keys, ks), 2), torch.cat((values, vs), 2)
        summary.update(first=old_cut // block)
        codes, scales = plain_summary(cache, block)
        assert (summary.codes[:, :, :summary.blocks].cpu().numpy() == codes).all()
        assert (summary.scales[:, :, :summary.blocks].cpu().numpy() == scales).all()


@pytest.mark.gpu
def test_a_step_captured_as_one_graph(kvq):  # noqa: F811
    """rope -> tree attention -> block choice -> block attention, replayed on new contents."""
    b, hq, hkv, n, t, d = 2, 16, 2, 960, 4, 128
    gen = torch.Generator(device="cuda").manual_seed(8)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    cache = kvq.pack(rand(b, hkv, n, d), rand(b, hkv, n, d), 128, "bf16")
    q, k, v = rand(b, hq, t, d), rand(b, hkv, t, d), rand(b, hkv, t, d)
    pos = (n + torch.arange(t, device="cuda", dtype=torch.int32)).expand(b, t).contiguous()
    par = torch.arange(-1, t - 1, dtype=torch.int32, device="cuda").expand(b, t).contiguous()
    rope = kvq.Rope(kvq.RopePlan(d), q, k, pos)
    tree = kvq.AttendTree(cache, rope.out[0], rope.out[1], v, par)
    summary = kvq.BlockSummary(cache, 32)
    sparse = kvq.AttendBlocks(cache, rope.out[0], summary, 5)

    def step():
        rope.run()
        tree.run()
        summary.update()
        sparse.run()

    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for x in (q, k, v):
        x.copy_(rand(*x.shape))
    pos.add_(3)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (tree.out, sparse.out, sparse.selected)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, (tree.out, sparse.out, sparse.selected)))
    compare(tree.out, plain(cache, kvq, rope.out[0], rope.out[1], v, par), par,
            TOL_TENSOR + 2.0 ** -8)


@pytest.mark.gpu
def test_offsets_past_32_bits(kvq):  # noqa: F811
    """The last (sequence, head) of a cache whose K and V codes pass 2^31 bytes each."""
    b, hkv, n, d = 5, 8, 900_000, 128     # 40 x 900,000 x 64 bytes = 2.3e9
    k = torch.zeros((b, hkv, n, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    gen = torch.Generator(device="cuda").manual_seed(2)
    k[-1, -1] = torch.randn((n, d), generator=gen, device="cuda").bfloat16()
    v[-1, -1] = torch.randn((n, d), generator=gen, device="cuda").bfloat16()
    cache = kvq.pack(k, v, 64, "bf16")
    k1, v1 = k[-1:, -1:].clone(), v[-1:, -1:].clone()
    del k, v
    one = kvq.pack(k1, v1, 64, "bf16")     # that head as a cache of its own
    kd, vd = dequant(one, kvq)
    t = 3
    q = torch.randn((b, 8 * hkv, t, d), generator=gen, device="cuda").bfloat16()
    kt = torch.randn((b, hkv, t, d), generator=gen, device="cuda").bfloat16()
    vt = torch.randn((b, hkv, t, d), generator=gen, device="cuda").bfloat16()
    par = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device="cuda").expand(b, t).contiguous()
    out, st = kvq.attend_tree(cache, q, kt, vt, par, out_dtype="f32")
    assert kvq.read_status(st) == 0
    seen = ancestors(par)[-1]
    for h in range(8 * (hkv - 1), 8 * hkv):
        kk = torch.cat((kd[0, 0], kt[-1, -1].double()))
        vv = torch.cat((vd[0, 0], vt[-1, -1].double()))
        s = q[-1, h].double() @ kk.T / d ** 0.5
        s[:, n:] = torch.where(seen, s[:, n:], -torch.inf)
        want = torch.softmax(s, 1) @ vv
        assert float((out[-1, h].double() - want).norm() / want.norm()) <= TOL_TENSOR
    big = kvq.BlockSummary(cache, 64).update()
    small = kvq.BlockSummary(one, 64).update()
    assert torch.equal(big.codes[-1, -1, :small.blocks], small.codes[0, 0, :small.blocks])
    assert torch.equal(big.values(small.blocks - 7)[-1, -1], small.values(small.blocks - 7)[0, 0])
    o1, s1, _ = kvq.attend_blocks(cache, q[:, :, :1], big, 12, n_sink=1, out_dtype="f32")
    o2, s2, _ = kvq.attend_blocks(one, q[-1:, -8:, :1].contiguous(), small, 12, n_sink=1,
                                  out_dtype="f32")
    assert torch.equal(s1[-1, -1], s2[0, 0])
    # the same keys in slices of other lengths: partial sums merge in another order
    assert float((o1[-1, -8:] - o2[0]).norm() / o2.norm()) <= 1e-3
