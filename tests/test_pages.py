"""The paged cache: its tables, the append of ragged rows, the read-back of tokens and
attention over the pages, against a host model of the rules (include/kvq.h) and the
64-bit oracle.

Tolerances. Values read back: code * scale is one fp32 product, rounded once to the
output's type (2^-24 in fp32, 2^-8 + 2^-24 in bf16, relative); a scale that were one
step off would show. Attention in fp32: a score of D products is off by at most
(D + 2) 2^-24 sum|q k| scale log2 e, below 1e-4 for the values here, and so is the
output (relative L2). On the tensor cores: q * scale, the K scales and their product,
the probabilities, the V scales and their product are each rounded to 11 bits (2^-11),
six roundings of 2^-11 in all: 3e-3 if all had one sign, held to 5e-3.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kvq_oracle as O  # noqa: E402

TOL_TENSOR, TOL_F32 = 5e-3, 1e-4


@pytest.fixture(scope="module")
def kvq():
    import os
    from quantized_sparse_kv_gb300 import build, kvq as k
    if not os.path.exists(k.LIB_PATH):
        build.build()
    k.load_library()
    return k


# ------------------------------------------------------------------ a host model
class Model:
    """The rules of kv_page_tables, request by request."""

    def __init__(self, slots, n_pages, page, max_pages, window):
        self.slots, self.page, self.max_pages, self.window = slots, page, max_pages, window
        self.free = list(range(n_pages))
        self.table = [[] for _ in range(slots)]
        self.length = [0] * slots

    def cut(self, n):
        return (n - self.window) // 32 * 32 if n >= self.window else 0

    def pages(self, n):
        return -(-self.cut(n) // self.page)

    def step(self, n_new, rows):
        """(offsets, before, after, row_slot, positions, work, flags); moves the state on."""
        flags, asked, first = 0, 0, 0
        before = list(self.length)
        offsets, slot, pos, work = [], [-1] * rows, [0] * rows, []
        for s, n in enumerate(n_new):
            if n == -1:
                self.free += self.table[s]
                self.table[s], self.length[s] = [], 0
        have = len(self.free)
        for s, n in enumerate(n_new):
            offsets.append(min(first, 2 ** 30))
            if n < -1:
                flags |= 1
            if n <= 0:
                continue
            first += n
            end = before[s] + n
            if first > rows:
                flags |= 1
                continue
            if self.pages(end) > self.max_pages:
                flags |= 16
                continue
            need = self.pages(end) - self.pages(before[s])
            asked += need
            if need and asked > have:
                flags |= 16
                continue
            self.table[s] += [self.free.pop() for _ in range(need)]
            self.length[s] = end
            for i in range(n):
                slot[offsets[s] + i], pos[offsets[s] + i] = s, before[s] + i
            c1 = self.cut(end) // 32
            work += [(s, g) for g in range(self.cut(before[s]) // 32, c1)]
            work += [(s, g) for g in range(max(before[s] // 32, c1), -(-end // 32))]
        offsets.append(min(first, 2 ** 30))
        return offsets, before, list(self.length), slot, pos, work, flags


def check_plan(kvq, state, model, plan, want):
    offsets, before, after, slot, pos, work, flags = want
    assert kvq.read_status(plan.status) == flags
    assert plan.offsets.tolist() == offsets
    assert plan.before.tolist() == before and plan.after.tolist() == after
    assert plan.row_slot.tolist() == slot and plan.positions.tolist() == pos
    n = int(plan.counts[1])
    got = plan.work[:n].tolist()
    assert [(w[0], w[1]) for w in got] == work
    table = state.table.tolist()
    for s, g, page, b, e, row, _, _ in got:
        assert (b, e, row) == (before[s], after[s], offsets[s])
        packed = g < model.cut(e) // 32
        assert page == (table[s][g * 32 // model.page] if packed else -1)
    assert int(plan.free_after) == len(model.free) and int(plan.counts[2]) == 0


def check_state(state, model):
    assert state.lengths.tolist() == model.length
    n = int(state.n_free[0])
    assert state.free_pages[:n].tolist() == model.free
    table = state.table.tolist()
    for s, pages in enumerate(model.table):
        assert table[s][:len(pages)] == pages, s


def sequence_values(model, tokens, s, wdt):
    """K and V of request s as attention reads them, [heads][length][D] in 64 bits."""
    k, v = tokens[s]
    n = k.shape[0]
    recent = n - model.cut(n)
    out = []
    for h in range(k.shape[1]):
        out.append(O.dequantize_head(O.pack_head(k[:, h], v[:, h], recent, wdt)))
    return np.stack([x[0] for x in out]), np.stack([x[1] for x in out])


def new_rows(gen, rows, heads, d, dt, wdt):
    """Rows for the GPU and what the cache keeps of them."""
    x = torch.randn((rows, heads, d), generator=gen, device="cuda").to(dt)
    kept = x.bfloat16() if wdt == "bf16" else x
    return x, kept.float().cpu().numpy()


def poison(cache):
    """No byte that was not written may reach a result: NaN in every type."""
    cache.pool.fill_(255)
    cache.ring.fill_(255)


def check_values(kvq, cache, model, tokens, wdt, out_dtype):
    slot = [s for s in range(model.slots) for _ in range(model.length[s])]
    pos = [p for s in range(model.slots) for p in range(model.length[s])]
    if not slot:
        return
    call = kvq.PageValues(cache, torch.tensor(slot, device="cuda"),
                          torch.tensor(pos, device="cuda"), out_dtype)
    got = [x.float().cpu().numpy() for x in call.run()]
    assert kvq.read_status(call.status) == 0
    tol = 2.0 ** -24 if out_dtype == "f32" else 2.0 ** -8 + 2.0 ** -24
    at = 0
    for s in range(model.slots):
        n = model.length[s]
        if n:
            for x, want in zip(got, sequence_values(model, tokens, s, wdt)):
                have = x[at:at + n].transpose(1, 0, 2)
                assert (np.abs(have - want) <= tol * np.abs(want)).all(), s
        at += n


def attention64(q, k, v):
    """q (heads, D) over k, v (kv_heads, n, D)."""
    group = q.shape[0] // k.shape[0]
    out = np.zeros(q.shape)
    for h in range(q.shape[0]):
        a = k[h // group] @ q[h] / np.sqrt(q.shape[1])
        p = np.exp(a - a.max())
        out[h] = (p / p.sum()) @ v[h // group]
    return out


def check_attention(kvq, cache, model, tokens, wdt, group, gen, tol, q_dt, rng, path=None):
    hk, d = cache.kv_heads, cache.head_dim
    live = [s for s in range(model.slots) if model.length[s]]
    slot = [-1] + [s for s in range(model.slots)] + live
    pos = [0] + [model.length[s] - 1 for s in range(model.slots)]
    pos += [int(rng.integers(0, model.length[s])) for s in live]
    q = torch.randn((len(slot), hk * group, d), generator=gen, device="cuda").to(q_dt)
    q[0] = float("nan")
    out = torch.full(q.shape, 7.0, device="cuda")
    n = 1 + model.slots
    calls = [kvq.AttendPages(cache, q[:n], torch.tensor(slot[:n], device="cuda"), out=out[:n])]
    if live:
        calls.append(kvq.AttendPages(
            cache, q[n:], torch.tensor(slot[n:], device="cuda"),
            torch.tensor(pos[n:], device="cuda"), out=out[n:]))
    for call in calls:
        call.run()
        assert kvq.read_status(call.status) == 0
        if path:
            assert call.path == path
    got, q64 = out.double().cpu().numpy(), q.double().cpu().numpy()
    assert (got[0] == 7.0).all()
    values = {s: sequence_values(model, tokens, s, wdt) for s in live}
    for i, (s, p) in enumerate(zip(slot, pos)):
        if s == -1:
            continue
        if not model.length[s]:
            assert (got[i] == 0.0).all()
            continue
        k, v = values[s]
        want = attention64(q64[i], k[:, :p + 1], v[:, :p + 1])
        assert O.rel_l2(got[i], want) <= tol, (i, s, p)


# ------------------------------------------------------------------ steps of a server
CASES = [
    # slots, pages, page, max_pages, window, kv_heads, group, D, windows, rows' type, q's type
    (5, 40, 64, 12, 128, 2, 8, 128, "bf16", "bf16", "bf16"),
    (7, 90, 32, 30, 33, 1, 5, 128, "bf16", "f32", "f32"),
    (3, 30, 128, 9, 100, 4, 16, 64, "bf16", "bf16", "bf16"),
    (4, 60, 32, 20, 0, 2, 1, 128, "bf16", "bf16", "bf16"),
    (4, 60, 64, 20, 1, 3, 7, 64, "bf16", "bf16", "f32"),
    (4, 30, 64, 20, 31, 2, 3, 96, "f32", "f32", "f32"),
    (3, 30, 32, 20, 65, 2, 9, 256, "bf16", "bf16", "bf16"),
    (3, 30, 64, 20, 64, 1, 2, 32, "f32", "bf16", "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("slots,pages,page,most,window,hk,group,d,wdt,in_dt,q_dt", CASES)
def test_steps(kvq, slots, pages, page, most, window, hk, group, d, wdt, in_dt, q_dt):
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    rng = np.random.default_rng(window + d)
    gen = torch.Generator(device="cuda").manual_seed(window + d)
    state = kvq.PageState(slots, pages, page, most, window)
    cache = kvq.PagedCache(state, hk, d, wdt)
    poison(cache)
    model = Model(slots, pages, page, most, window)
    tokens = [None] * slots
    tensor = d in (64, 128) and wdt == "bf16"
    seen_full = False
    for step in range(14):
        n_new = []
        for s in range(slots):
            kind = rng.integers(0, 8)
            if model.length[s] == 0 or kind == 0:
                n = int(rng.integers(0, 500))
            elif kind == 1:
                n = -1 if step > 3 else 2
            elif kind == 2:
                n = 0
            elif kind == 3:
                n = int(rng.integers(1, 150))
            else:
                n = 1
            n_new.append(n)
        rows = sum(max(0, n) for n in n_new) + int(rng.integers(0, 3))
        k, kept_k = new_rows(gen, rows, hk, d, types[in_dt], wdt)
        v, kept_v = new_rows(gen, rows, hk, d, types[in_dt], wdt)
        new = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        look = kvq.PageTables(state, new, rows).run(advance=False)
        check_state(state, model)
        plan = kvq.PageTables(state, new, rows).run()
        want = model.step(n_new, rows)
        seen_full |= bool(want[-1] & 16)
        check_plan(kvq, state, model, plan, want)
        check_plan(kvq, state, model, look, want)
        check_state(state, model)
        call = kvq.AppendPages(cache, plan, k, v)
        call.run()
        assert kvq.read_status(call.status) == 0
        for s in range(slots):
            if model.length[s] == 0:
                tokens[s] = None
            elif model.length[s] > want[1][s]:
                lo = want[0][s]
                add = [x[lo:lo + n_new[s]] for x in (kept_k, kept_v)]
                tokens[s] = add if not want[1][s] else [np.concatenate(x)
                                                        for x in zip(tokens[s], add)]
        if step % 3 == 2 or step == 13:
            check_values(kvq, cache, model, tokens, wdt, "f32" if step % 2 else "bf16")
            check_attention(kvq, cache, model, tokens, wdt, group, gen,
                            TOL_TENSOR if tensor else TOL_F32, types[q_dt], rng,
                            "pages_tensor" if tensor else "pages_rows")
    assert max(model.length) > 200


@pytest.mark.gpu
def test_requests_that_get_nothing(kvq):
    # 10 pages of 32, at most 6 a request, window 0: 32 tokens a page
    state = kvq.PageState(6, 10, 32, 6, 0)
    model = Model(6, 10, 32, 6, 0)

    def go(n_new, rows):
        new = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        plan = kvq.PageTables(state, new, rows).run()
        check_plan(kvq, state, model, plan, model.step(n_new, rows))
        check_state(state, model)

    go([64, 0, 31, 160, 5, 0], 260)
    go([32 * 5, 1, 1, 1, 1, 1], 165)      # request 0 asks for more pages than one may have
    go([0, 96, 1, 32, 1, 31], 161)        # 2 pages are left: 1 gets none, 3 neither, 4 goes on
    go([0, 33, -1, -5, 2, 40], 50)        # ended, below -1, more rows than there are
    go([-1, 33, 0, -1, -1, 1], 34)
    go([0] * 6, 0)
    go([2 ** 31 - 1, 1, 1, 2 ** 28, 0, 0], 5)
    state.lengths[1] = -3                  # lengths that no table holds: left alone
    state.lengths[2] = 32 * 6 + 32
    new = torch.tensor([1, 1, 1, 1, 0, 0], dtype=torch.int32, device="cuda")
    plan = kvq.PageTables(state, new, 4).run()
    assert kvq.read_status(plan.status) == kvq.DEV_INDEX
    assert state.lengths.tolist()[1:3] == [-3, 224]
    assert plan.row_slot.tolist() == [0, -1, -1, 3]


@pytest.mark.gpu
@pytest.mark.parametrize("slots", [1, 300, 1025, 8192])
def test_many_slots(kvq, slots):
    rng = np.random.default_rng(slots)
    n_pages = 4 * slots
    state = kvq.PageState(slots, n_pages, 32, 9, 40)
    model = Model(slots, n_pages, 32, 9, 40)
    for step in range(4):
        n_new = [int(n) for n in rng.choice([0, 1, 1, 1, 70, 150, -1], slots)]
        rows = sum(max(0, n) for n in n_new) + 5
        new = torch.tensor(n_new, dtype=torch.int64, device="cuda")
        plan = kvq.PageTables(state, new, rows).run()
        check_plan(kvq, state, model, plan, model.step(n_new, rows))
        check_state(state, model)


@pytest.mark.gpu
def test_a_captured_step_serves_all_steps(kvq):
    """Tables, positions, append and attention of a decoding step in one graph."""
    slots, hk, hq, d, window = 6, 2, 16, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    state = kvq.PageState(slots, 80, 32, 20, window)
    layers = [kvq.PagedCache(state, hk, d) for _ in range(2)]
    model = Model(slots, 80, 32, 20, window)
    lengths = [63, 95, 200, 1, 127, 0]
    tokens = [[None] * slots for _ in layers]
    rows = sum(lengths)
    plan = kvq.page_tables(state, torch.tensor(lengths, device="cuda"), rows)
    model.step(lengths, rows)
    for cache, mine in zip(layers, tokens):
        poison(cache)
        k, kept_k = new_rows(gen, rows, hk, d, torch.bfloat16, "bf16")
        v, kept_v = new_rows(gen, rows, hk, d, torch.bfloat16, "bf16")
        kvq.append_pages(cache, plan, k, v)
        for s in range(slots):
            lo = sum(lengths[:s])
            mine[s] = [kept_k[lo:lo + lengths[s]], kept_v[lo:lo + lengths[s]]]
    rope = kvq.RopePlan(d)
    x = torch.zeros((8, hq + 2 * hk, d), dtype=torch.bfloat16, device="cuda")
    n_new = torch.zeros(slots, dtype=torch.int32, device="cuda")
    step = kvq.PageTables(state, n_new, 8)
    turn = kvq.Rope(rope, x[:, :hq].unsqueeze(2), x[:, hq:hq + hk].unsqueeze(2),
                    step.positions.view(8, 1), v=x[:, hq + hk:].unsqueeze(2))
    calls = [(kvq.AppendPages(c, step, turn.out[1].squeeze(2), turn.out[2].squeeze(2)),
              kvq.AttendPages(c, turn.out[0].squeeze(2), step.row_slot)) for c in layers]

    def one():
        step.run()
        turn.run()
        for put, get in calls:
            put.run()
            get.run()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()       # n_new is zero: nothing moves
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    rng = np.random.default_rng(3)
    for t in range(40):
        add = [int(v) for v in rng.choice([0, 1, 1, 1], slots)]
        if t % 9 == 5:
            add[int(rng.integers(slots))] = 3
        add = add if sum(add) <= 8 else [1] * slots
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        n_new.copy_(torch.tensor(add))
        graph.replay()
        torch.cuda.synchronize()
        want = model.step(add, 8)
        check_plan(kvq, state, model, step, want)
        check_state(state, model)
        for (put, get), cache, mine in zip(calls, layers, tokens):
            for s in range(slots):
                if add[s]:
                    lo = want[0][s]
                    new = [y[lo:lo + add[s], :, 0].float().cpu().numpy() for y in turn.out[1:]]
                    mine[s] = [np.concatenate(z) for z in zip(mine[s], new)]
            if t % 10 == 9:
                check_values(kvq, cache, model, mine, "bf16", "f32")
                got, q64 = get.out.double().cpu().numpy(), turn.out[0].double().cpu().numpy()
                for i, s in enumerate(want[3]):
                    if s >= 0:
                        k, v = sequence_values(model, mine, s, "bf16")
                        ref = attention64(q64[i, :, 0], k, v)
                        assert O.rel_l2(got[i], ref) <= TOL_TENSOR
            assert kvq.read_status(put.status) == 0 and kvq.read_status(get.status) == 0


@pytest.mark.gpu
def test_strided_rows_and_another_stream(kvq):
    d, hk = 128, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    outs = []
    x = torch.randn((300, 3 * hk, d + 8), generator=gen, device="cuda").bfloat16()
    for how in range(3):
        state = kvq.PageState(2, 20, 32, 10, 32)
        cache = kvq.PagedCache(state, hk, d)
        poison(cache)
        k, v = x[:, :hk, :d], x[:, 2 * hk:, 8:]
        if how == 1:
            k, v = k.contiguous(), v.contiguous()
        if how == 2:  # rows that start between 16-byte boundaries
            y = torch.empty((300, 3 * hk, d + 9), dtype=torch.bfloat16, device="cuda")
            y[:, :, 1:] = x
            k, v = y[:, :hk, 1:d + 1], y[:, 2 * hk:, 9:]
        stream = torch.cuda.Stream() if how else torch.cuda.current_stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            plan = kvq.page_tables(state, torch.tensor([180, 120], device="cuda"), 300)
            kvq.append_pages(cache, plan, k, v)
            q = x[:7, :, :d][:, :1].expand(7, 4, d)
            out, status = kvq.attend_pages(cache, q, plan.row_slot[100:107],
                                           plan.positions[100:107])
            val = kvq.page_values(cache, plan.row_slot, plan.positions)
        stream.synchronize()
        assert int(status[0]) == 0
        outs.append([out, *val])
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(128, "bf16"), (32, "f32")])
def test_rows_and_pages_that_do_not_exist(kvq, d, wdt):
    gen = torch.Generator(device="cuda").manual_seed(9)
    state = kvq.PageState(3, 20, 32, 6, 10)
    cache = kvq.PagedCache(state, 1, d, wdt)
    poison(cache)
    k = torch.randn((200, 1, d), generator=gen, device="cuda")
    v = torch.randn((200, 1, d), generator=gen, device="cuda")
    plan = kvq.page_tables(state, torch.tensor([150, 50, 0], device="cuda"), 200)
    kvq.append_pages(cache, plan, k, v)
    q = torch.randn((6, 4, d), generator=gen, device="cuda")
    slot = torch.tensor([0, 3, -2, 1, 1, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([149, 0, 0, 50, -1, 0], dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 3.0, device="cuda")
    call = kvq.AttendPages(cache, q, slot, pos, out=out)
    call.run()
    assert kvq.read_status(call.status) == kvq.DEV_INDEX
    assert bool((out[1:] == 3.0).all()) and bool((out[0] != 3.0).all())
    vals = kvq.PageValues(cache, slot, pos)
    vals.k.fill_(3.0)
    vals.run()
    assert kvq.read_status(vals.status) == kvq.DEV_INDEX
    assert bool((vals.k[1:] == 3.0).all())
    # a page outside the pool: its tokens are skipped, those of the others stay
    good = int(state.table[0, 1])
    for bad in (-1, 20, 1 << 30):
        state.table[0, 1] = bad
        call = kvq.AttendPages(cache, q[:1], slot[:1], out_dtype="f32")
        got = call.run().double().cpu().numpy()[0]
        assert kvq.read_status(call.status) == kvq.DEV_INDEX
        model = Model(3, 20, 32, 6, 10)
        kept = [k[:150].float().cpu().numpy(), v[:150].float().cpu().numpy()]
        if wdt == "bf16":
            kept = [O.round_to_bf16(x) for x in kept]
        kk, vv = sequence_values(model, [kept], 0, wdt)
        keep = np.r_[0:32, 64:150]
        want = attention64(q[0].double().cpu().numpy(), kk[:, keep], vv[:, keep])
        assert O.rel_l2(got, want) <= TOL_TENSOR
    state.table[0, 1] = good
    # pages outside the pool that a broken table or free list brings into a step
    for bad in (-1, 20, 1 << 30):
        state.free_pages.fill_(bad)
        step = kvq.page_tables(state, torch.tensor([0, 0, 100], device="cuda"), 100)
        again = kvq.AppendPages(cache, step, k[:100], v[:100])
        again.run()
        assert kvq.read_status(again.status) == kvq.DEV_INDEX
        kvq.page_tables(state, torch.tensor([0, 0, -1], device="cuda"), 0)


# ------------------------------------------------------------------ refusals (no GPU)
ADDR = 1 << 20


def host_state(kvq, **kw):
    f = dict(slots=4, n_pages=10, page=64, max_pages=5, window=128, table=ADDR, lengths=ADDR,
             free_pages=ADDR, n_free=ADDR)
    f.update(kw)
    return kvq.KvqPageState(*f.values())


def host_cache(kvq, state=None, **kw):
    f = dict(kv_heads=2, head_dim=128, win_dtype=1, pool=ADDR, ring=ADDR)
    f.update(kw)
    return kvq.KvqPagedCache(state or host_state(kvq), *f.values())


def host_plan(kvq, rows=10, cap=None, **kw):
    f = dict(offsets=ADDR, before=ADDR, after=ADDR, row_slot=ADDR, positions=ADDR, work=ADDR,
             counts=ADDR)
    f.update(kw)
    return kvq.KvqPagePlan(rows, 1000 if cap is None else cap, *f.values())


BAD_STATES = [dict(slots=0), dict(slots=8193), dict(n_pages=0), dict(n_pages=(1 << 28) + 1), dict(page=16), dict(page=96),
              dict(max_pages=0), dict(window=-1), dict(window=65537), dict(max_pages=1 << 26)]


@pytest.mark.parametrize("kw", BAD_STATES)
def test_states_that_are_refused(kvq, kw):
    lib = kvq.load_library()
    sizes = (ctypes.c_size_t * 6)()
    state = host_state(kvq, **kw)
    r = ctypes.byref
    assert lib.kvq_paged_sizes(r(host_cache(kvq, state)), sizes) == 1
    assert lib.kvq_page_work(r(state), 5) == 0
    assert lib.kv_page_tables(r(state), ADDR, r(host_plan(kvq)), 1, None, None) == 1


def test_sizes(kvq):
    lib = kvq.load_library()
    sizes = (ctypes.c_size_t * 6)()
    assert lib.kvq_paged_sizes(ctypes.byref(host_cache(kvq)), sizes) == 0
    # window 128: (128 + 63) // 32 = 5 tiles
    assert list(sizes) == [4 * 4 * 5, 16, 40, 16, 10 * 2 * 2 * 5120, 4 * 2 * 5 * 2 * 32 * 128 * 2]
    for kw in (dict(kv_heads=0), dict(head_dim=48), dict(head_dim=288), dict(win_dtype=2)):
        assert lib.kvq_paged_sizes(ctypes.byref(host_cache(kvq, **kw)), sizes) == 1
    assert lib.kvq_page_work(ctypes.byref(host_state(kvq)), 0) == 0
    assert lib.kvq_page_work(ctypes.byref(host_state(kvq)), -1) == 0
    assert lib.kvq_page_work(ctypes.byref(host_state(kvq)), (1 << 28) + 1) == 0


def test_work_bound_holds_every_step(kvq):
    # the groups of a step by the host model, over windows, lengths and new tokens
    lib = kvq.load_library()
    rng = np.random.default_rng(0)
    for window in (0, 1, 31, 32, 33, 64, 97, 128, 200):
        for _ in range(300):
            slots = int(rng.integers(1, 4))
            m = Model(slots, 10 ** 6, 32, 10 ** 5, window)
            m.length = [int(x) for x in rng.integers(0, 500, slots)]
            m.table = [[0] * m.pages(n) for n in m.length]
            n_new = [int(x) for x in rng.choice([0, 1, 2, 31, 32, 33, 64, 95, 129, 300], slots)]
            work = m.step(n_new, sum(n_new))[5]
            st = host_state(kvq, slots=slots, n_pages=10 ** 6, page=32, max_pages=10 ** 5,
                            window=window)
            assert len(work) <= lib.kvq_page_work(ctypes.byref(st), sum(n_new))


def test_pointers_and_arguments_that_are_refused(kvq):
    lib, r = kvq.load_library(), ctypes.byref
    st, c, p = host_state(kvq), host_cache(kvq), host_plan(kvq)
    arg, align, space, unsup = 1, 2, 4, 3
    for name in ("table", "lengths", "free_pages", "n_free"):
        assert lib.kv_page_tables(r(host_state(kvq, **{name: None})), ADDR, r(p), 1, None, None) == arg
        assert lib.kv_page_tables(r(host_state(kvq, **{name: ADDR + 4})), ADDR, r(p), 1, None,
                                  None) == align
    assert lib.kv_page_tables(None, ADDR, r(p), 1, None, None) == arg
    assert lib.kv_page_tables(r(st), None, r(p), 1, None, None) == arg
    assert lib.kv_page_tables(r(st), ADDR, None, 1, None, None) == arg
    assert lib.kv_page_tables(r(st), ADDR, r(p), 1, ADDR + 4, None) == align
    for name in ("offsets", "before", "after", "row_slot", "positions", "work", "counts"):
        assert lib.kv_page_tables(r(st), ADDR, r(host_plan(kvq, **{name: None})), 1, None, None) == arg
        assert lib.kv_page_tables(r(st), ADDR, r(host_plan(kvq, **{name: ADDR + 8})), 1, None,
                                  None) == align
    assert lib.kv_page_tables(r(st), ADDR, r(host_plan(kvq, rows=-1)), 1, None, None) == arg
    assert lib.kv_page_tables(r(st), ADDR, r(host_plan(kvq, rows=(1 << 28) + 1)), 1, None, None) == arg
    assert lib.kv_page_tables(r(st), ADDR, r(host_plan(kvq, cap=5)), 1, None, None) == space
    assert lib.kv_page_tables(r(st), ADDR, r(host_plan(kvq, cap=-1)), 1, None, None) == arg

    def rows(k=ADDR, v=ADDR, *strides):
        return kvq.KvqPageRows(k, v, *(strides or (256, 128, 256, 128)))

    def put(cache=c, plan=p, x=None, dt=1, status=None):
        return lib.kv_append_pages(r(cache), r(plan), r(x or rows()), dt, status, None)

    assert put(dt=2) == arg and put(x=rows(None)) == arg and put(x=rows(ADDR, None)) == arg
    assert put(x=rows(ADDR + 2)) == align and put(x=rows(ADDR, ADDR, 4, 128, 256, 128)) == align
    assert put(x=rows(ADDR, ADDR, -8, 128, 256, 128)) == arg
    assert put(cache=host_cache(kvq, pool=None)) == arg
    assert put(cache=host_cache(kvq, ring=ADDR + 8)) == align
    assert put(plan=host_plan(kvq, cap=1 << 30), cache=host_cache(kvq, kv_heads=4)) == unsup
    assert put(plan=host_plan(kvq, rows=0, row_slot=None, positions=None, work=None)) == 0

    def values(n=4, slot=ADDR, pos=ADDR, k=ADDR, v=ADDR, dt=0):
        return lib.kv_page_values(r(c), slot, pos, n, k, v, dt, None, None)

    assert values(n=-1) == arg and values(n=(1 << 28) + 1) == arg and values(dt=2) == arg
    assert values(slot=None) == arg and values(k=None) == arg and values(v=ADDR + 4) == align
    assert values(n=0, slot=None, pos=None, k=None, v=None) == 0

    sz = ctypes.c_size_t(1 << 40)

    def attend(cache=c, q=ADDR, q_dt=1, hq=16, n=4, slot=ADDR, pos=ADDR, out=ADDR, out_dt=1,
               ws=ADDR, size=sz):
        return lib.kv_attend_pages(r(cache), q, q_dt, hq, n, slot, pos, 0.0, out, out_dt, ws,
                                   r(size) if size is not None else None, None, None)

    assert attend(hq=15) == arg and attend(hq=0) == arg and attend(n=-1) == arg
    assert attend(n=65536) == arg and attend(n=5, slot=None) == arg and attend(q_dt=2) == arg
    assert attend(out_dt=2) == arg and attend(size=None) == arg
    assert attend(hq=65536) == unsup
    assert attend(size=ctypes.c_size_t(16)) == space
    assert attend(q=None) == arg and attend(out=None) == arg
    assert attend(q=ADDR + 2) == align and attend(pos=ADDR + 4) == align
    assert attend(ws=ADDR + 8) == align and attend(n=0, q=None, out=None) == 0


@pytest.mark.gpu
def test_the_binding_refuses(kvq):
    state = kvq.PageState(2, 4, 32, 4, 0)
    cache = kvq.PagedCache(state, 2, 64)
    other = kvq.PageState(2, 4, 32, 4, 0)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    plan = kvq.PageTables(state, n, 3)
    x = torch.zeros((3, 2, 64), device="cuda")
    for bad in (n.float(), n.bool()):
        with pytest.raises(TypeError):
            kvq.PageTables(state, bad, 3)
    with pytest.raises(ValueError):
        kvq.PageTables(state, n[:1], 3)
    with pytest.raises(ValueError):
        kvq.PageTables(state, n, -1)
    with pytest.raises(ValueError):
        kvq.PageTables(state, n.cpu(), 3)
    with pytest.raises(ValueError):
        kvq.AppendPages(cache, kvq.PageTables(other, n, 3), x, x)
    with pytest.raises(ValueError):
        kvq.AppendPages(cache, plan, x[:2], x[:2])
    with pytest.raises(TypeError):
        kvq.AppendPages(cache, plan, x, x.bfloat16())
    with pytest.raises(TypeError):
        kvq.AppendPages(cache, plan, x.half(), x.half())
    with pytest.raises(TypeError):
        kvq.AttendPages(cache, x.half())
    with pytest.raises(ValueError):
        kvq.AttendPages(cache, x[:, :, :32])
    with pytest.raises(kvq.KvqError):
        kvq.AttendPages(cache, x)  # three rows, two requests
    with pytest.raises(kvq.KvqError):
        kvq.AttendPages(cache, x[:2, :1], n)  # one query head, two KV heads
    with pytest.raises(TypeError):
        kvq.AttendPages(cache, x[:2], n.float())
    with pytest.raises(ValueError):
        kvq.AttendPages(cache, x[:2], n, n[:1])
    with pytest.raises(ValueError):
        kvq.AttendPages(cache, x[:2], n, out=x)
    with pytest.raises(ValueError):
        kvq.PageValues(cache, n, n[:1])
    with pytest.raises(ValueError):
        state.restore(lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(kvq.KvqError):
        kvq.PageState(2, 4, 48, 4, 0)
    # nothing to do is done
    assert kvq.attend_pages(cache, x[:0], n[:0])[0].shape == (0, 2, 64)
    empty = kvq.page_tables(state, n, 0)
    kvq.append_pages(cache, empty, x[:0], x[:0])
    assert kvq.page_values(cache, n[:0], n[:0])[0].shape == (0, 2, 64)
