"""The paged cache of requests of different lengths: tables built on the GPU, the append of
ragged rows, the read-back of listed tokens and the attention of new tokens over the
pages. The cases they are timed on, their inputs and their plain forms.

``run`` computes an operator with elementary torch operations in fp32 while
``own`` is false, and with the library's calls when it is true; ``exact``
computes the same outputs from the definitions, in fp64.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ cases


def listed():
    return [
        # the tables of one decoding step of a full batch: latency
        dict(name="tables_decode_b64", op="tables", slots=64, longest=32768, page=64, window=128,
             prompts=0, prompt=0, idle=4, leave=0),
        # a large server's step: most requests decode, some prompts come in, some requests leave
        dict(name="tables_mixed_b1024", op="tables", slots=1024, longest=8192, page=32, window=128,
             prompts=24, prompt=4096, idle=100, leave=40),
        # a decoding step's tokens into the cache: latency; some requests complete a group
        dict(name="append_decode_b64", op="append", slots=64, longest=4096, page=64, window=128,
             prompts=0, prompt=0, idle=0, kv_heads=2, head_dim=128, dtype="bf16", rows=True),
        # a step with prompts beside decoding requests, rows of the projection read in place
        dict(name="append_mixed_prompts", op="append", slots=48, longest=2048, page=64, window=128,
             prompts=10, prompt=16384, idle=3, kv_heads=2, head_dim=128, dtype="bf16", rows=True),
        # prompts of odd lengths in fp32 with fp32 windows, another head dim and an odd window
        dict(name="append_prompt_f32", op="append", slots=5, longest=700, page=32, window=33,
             prompts=3, prompt=1501, idle=1, kv_heads=4, head_dim=64, dtype="f32", rows=False),
        # a long request's cached prefix read back
        dict(name="values_prefix_16k", op="values", slots=2, longest=16384, page=64, window=128,
             rows=16384, order="prefix", kv_heads=2, head_dim=128),
        # tokens here and there over many requests
        dict(name="values_scattered", op="values", slots=37, longest=3001, page=32, window=100,
             rows=4099, order="any", kv_heads=2, head_dim=128),
        # one short request decoding: latency
        dict(name="attend_b1", op="attend", slots=1, rows=1, shortest=700, longest=700, page=64,
             window=128, kv_heads=2, group=8, head_dim=128, pad=0, each=1),
        # a batch of ragged medium contexts, padded to a captured size
        dict(name="attend_b29_ragged", op="attend", slots=40, rows=29, shortest=1, longest=4096,
             page=32, window=128, kv_heads=8, group=4, head_dim=128, pad=3, each=1),
        # the largest decode batch, long contexts
        dict(name="attend_b64_32k", op="attend", slots=64, rows=64, shortest=16384, longest=32768,
             page=64, window=128, kv_heads=2, group=8, head_dim=128, pad=0, each=1),
        # few very long contexts
        dict(name="attend_b8_128k", op="attend", slots=8, rows=8, shortest=100000, longest=131072,
             page=128, window=128, kv_heads=2, group=8, head_dim=128, pad=0, each=1),
        # several new tokens a request, each seeing those before it; a smaller head
        dict(name="attend_b12_each3", op="attend", slots=12, rows=36, shortest=300, longest=8191,
             page=64, window=100, kv_heads=4, group=7, head_dim=64, pad=0, each=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "values", "attend", "attend", "attend",
                     "attend"])
    page = rng.choice([32, 64, 64, 128])
    window = rng.choice([128, 128, rng.randint(1, 200)])
    if op == "tables":
        slots = _log(rng, 1, 2048)
        return dict(op=op, slots=slots, longest=_log(rng, 300, 32768 if slots < 300 else 8192),
                    page=page, window=window, prompts=rng.randint(0, min(24, slots // 3)),
                    prompt=_log(rng, 1, 4096), idle=rng.randint(0, slots // 3),
                    leave=rng.randint(0, slots // 4))
    if op == "append":
        slots = _log(rng, 1, 64)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        return dict(op=op, slots=slots, longest=_log(rng, 130, 4096), page=page, window=window,
                    prompts=rng.randint(0, min(8, slots)), prompt=_log(rng, 1, 4096),
                    idle=rng.randint(0, slots // 4), kv_heads=rng.choice([1, 2, 2, 4]),
                    head_dim=rng.choice([64, 128, 128]), dtype=dtype, rows=rng.random() < 0.5)
    if op == "values":
        return dict(op=op, slots=_log(rng, 1, 64), longest=_log(rng, 200, 8192), page=page,
                    window=window, rows=_log(rng, 1, 16384), order=rng.choice(["prefix", "any"]),
                    kv_heads=rng.choice([1, 2, 4]), head_dim=rng.choice([64, 128]))
    kv_heads, group = rng.choice([(2, 8), (2, 8), (8, 4), (1, 7), (4, 5), (2, 16), (8, 1)])
    longest = _log(rng, 100, 131072)
    each = rng.choice([1, 1, 1, 2, 4])
    slots = _log(rng, 1, 64)
    while slots * longest * kv_heads > 64 * 32768 * 2 or (slots * longest * kv_heads * each
                                                          > 64 * 24576 * 2):
        slots -= 1
        if slots < 1:
            slots, longest = 1, longest // 2
    return dict(op=op, slots=slots, rows=each * rng.randint((slots + 1) // 2, slots),
                shortest=max(each, longest // rng.choice([1, 2, 50])), longest=max(each, longest),
                page=page, window=window, kv_heads=kv_heads, group=group,
                head_dim=rng.choice([128, 128, 64]), pad=rng.choice([0, 0, 2]), each=each)


# ------------------------------------------------------------------ the layout's arithmetic


def _cut(length, window):
    """Tokens held as int4 of a request of this length (numbers or tensors)."""
    if isinstance(length, int):
        return (length - window) // 32 * 32 if length >= window else 0
    return torch.div((length - window).clamp(min=0), 32, rounding_mode="floor") * 32


def _pages(length, window, page):
    return (_cut(length, window) + page - 1) // page


def _cap(window):
    """Window rows of a request: a ring, row = position modulo this."""
    return (window + 63) // 32 * 32


def _rows(case):
    """Token rows of the largest step of a case: one of each decoding request, all prompts."""
    rest = case["slots"] - case["prompts"] - case["idle"] - case.get("leave", 0)
    return case["prompts"] * max(1, case["prompt"]) + max(0, rest)


def _host(gen, lo, hi, n):
    """n whole numbers in [lo, hi], on the host."""
    return torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda").tolist()


# ------------------------------------------------------------------ inputs


def _keys(gen, shape, gain):
    """Keys with a few strong channels, as trained keys have them."""
    return torch.randn(shape, generator=gen, device="cuda").mul_(gain)


def _gain(gen, kv_heads, d):
    g = 0.5 + torch.rand((kv_heads, d), generator=gen, device="cuda")
    return g * torch.where(torch.rand((kv_heads, d), generator=gen, device="cuda") < 0.03,
                           4.0, 1.0)


def _over_7(x):
    """x / 7, correctly rounded (a division by a number would multiply by its reciprocal)."""
    return x / torch.full_like(x, 7.0)


def _quantize(x, dim):
    """int4 codes and scales, one scale per group along `dim` (32 long)."""
    scale = _over_7(x.abs().amax(dim, keepdim=True))
    code = torch.where(scale > 0, torch.round(x / scale), torch.zeros_like(x)).clamp_(-7, 7)
    return code.to(torch.int8), scale.squeeze(dim)


def _plain_cache(case, slots, pages):
    """Pages in an order of their own, a page for what is not kept, and empty windows."""
    h, d, page = case["kv_heads"], case["head_dim"], case["page"]
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    dev = "cuda"
    return dict(
        k_codes=torch.zeros((pages + 1, h, page, d), dtype=torch.int8, device=dev),
        k_scales=torch.zeros((pages + 1, h, page // 32, d), device=dev),
        v_codes=torch.zeros((pages + 1, h, page, d), dtype=torch.int8, device=dev),
        v_scales=torch.zeros((pages + 1, h, page, d // 32), device=dev),
        k_ring=torch.zeros((slots, h, _cap(case["window"]), d), dtype=dt, device=dev),
        v_ring=torch.zeros((slots, h, _cap(case["window"]), d), dtype=dt, device=dev))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, window, page, slots = case["op"], case["window"], case["page"], case["slots"]
    s = dict(case=case)
    # lengths before the step, and what each request brings: 1 token, a prompt, none, or -1
    # (those of an append are the case's own: they say how many values come back)
    own_gen = gen
    if op == "append":
        gen = torch.Generator(device="cuda")
        gen.manual_seed(slots)
    before = _host(gen, case.get("shortest", 1), case["longest"], slots)
    if op in ("tables", "append"):
        step = [1] * slots
        at = torch.randperm(slots, generator=gen, device="cuda").tolist()
        sizes = _host(gen, max(1, case["prompt"] // 2), max(1, case["prompt"]), slots)
        for i in at[:case["prompts"]]:
            before[i], step[i] = 0, sizes[i]
        rest = at[case["prompts"]:]
        for i in rest[:case["idle"]]:
            step[i] = 0
        for i in rest[case["idle"]:case["idle"] + case.get("leave", 0)]:
            step[i] = -1
        after = [0 if n < 0 else b + n for b, n in zip(before, step)]
        rows = sum(n for n in step if n > 0)
        if op == "tables":  # the step's tensors are as large as the largest such step
            rows = _rows(case)
        s["rows"] = rows
    else:
        before[0] = case["longest"]
        step, after = [0] * slots, before
    gen = own_gen
    held = [_pages(b, window, page) for b in before]
    need = [max(0, _pages(a, window, page) - p) for a, p in zip(after, held)]
    most = max(1, _pages(max(case["longest"] + 1, case.get("prompt", 0)), window, page))
    total = slots * most + 5
    order = torch.randperm(total, generator=gen, device="cuda")
    table = torch.full((slots, most), -1, dtype=torch.int32)
    free = order.to(torch.int32).cpu()
    used = 0
    for i, p in enumerate(held):
        table[i, :p] = free[used:used + p]
        used += p
    free = torch.cat((free[used:], torch.full((used,), -1, dtype=torch.int32)))
    s.update(table=table.cuda(), free=free.cuda(),
             n_free=torch.tensor([total - used, 0, 0, 0], dtype=torch.int32, device="cuda"),
             lengths=torch.tensor(before, dtype=torch.int32, device="cuda"),
             n_new=torch.tensor(step, dtype=torch.int32, device="cuda"), total=total)
    if op == "tables":
        if own:
            from quantized_sparse_kv_gb300 import kvq
            state = kvq.PageState(slots, total, page, max_pages=most, window=window)
            state.restore(s["table"], s["lengths"], s["free"], s["n_free"])
            s["call"] = kvq.PageTables(state, s["n_new"], rows)
        return s

    # the cache's contents: every request's tokens
    h, d = case["kv_heads"], case["head_dim"]
    f32 = case.get("dtype") == "f32"
    dt = torch.float32 if f32 else torch.bfloat16
    gain = _gain(gen, h, d)
    if own:
        from quantized_sparse_kv_gb300 import kvq
        state = kvq.PageState(slots, total, page, max_pages=most, window=window)
        state.restore(None, None, torch.randperm(total, device="cuda"), None)
        s["cache"] = cache = kvq.PagedCache(state, h, d, "f32" if f32 else "bf16")
    else:
        s["cache"] = c = _plain_cache(case, slots, total)
        cap, bins = _cap(window), -(-max(max(before), 1) // page)
    widest = max(max(before), 1)
    stepping = max(1, (1 << 27) // (widest * h * d))  # requests made at a time
    for b0 in range(0, slots, stepping):
        b1 = min(slots, b0 + stepping)
        n = torch.tensor(before[b0:b1], device="cuda")
        k = _keys(gen, (b1 - b0, widest, h, d), gain).to(dt)
        v = torch.randn((b1 - b0, widest, h, d), generator=gen, device="cuda").to(dt)
        there = torch.arange(widest, device="cuda") < n[:, None]
        if own:
            if int(n.sum()):
                new = torch.zeros(slots, dtype=torch.int32, device="cuda")
                new[b0:b1] = n
                plan = kvq.page_tables(state, new, int(n.sum()))
                kvq.append_pages(cache, plan, k[there], v[there])
            continue
        cut = _cut(n, window)
        kept = (torch.arange(bins * page, device="cuda") < cut[:, None])
        pad = (0, 0, 0, 0, 0, bins * page - widest)
        kq = torch.nn.functional.pad(k.float(), pad)
        vq = torch.nn.functional.pad(v.float(), pad)
        kc, ks = _quantize(kq.view(b1 - b0, bins * page // 32, 32, h, d), 2)
        vc, vs = _quantize(vq.view(b1 - b0, bins * page, h, d // 32, 32), 4)
        tab = torch.full((b1 - b0, bins), total, dtype=torch.long, device="cuda")
        wide = min(bins, most)
        held_t = kept.view(b1 - b0, bins, page)[:, :wide, 0]
        tab[:, :wide] = torch.where(held_t, s["table"][b0:b1, :wide].long(), total)
        c["k_codes"][tab] = kc.view(b1 - b0, bins, page, h, d).transpose(2, 3)
        c["k_scales"][tab] = ks.view(b1 - b0, bins, page // 32, h, d).transpose(2, 3)
        c["v_codes"][tab] = vc.view(b1 - b0, bins, page, h, d).transpose(2, 3)
        c["v_scales"][tab] = vs.view(b1 - b0, bins, page, h, d // 32).transpose(2, 3)
        w = torch.arange(cap, device="cuda")
        pos = cut[:, None] + (w - cut[:, None]) % cap
        row = torch.arange(b1 - b0, device="cuda")[:, None]
        live = (pos < n[:, None])[:, :, None, None]
        pos = pos.clamp(max=widest - 1)
        for ring, x in (("k_ring", k), ("v_ring", v)):
            c[ring][b0:b1] = torch.where(live, x[row, pos], c[ring].new_zeros(())).transpose(1, 2)
    del k, v

    if op == "append":
        if case["rows"]:  # one row per token: four query heads a KV head, k heads, v heads
            x = torch.randn((rows, 6 * h, d), generator=gen, device="cuda")
            x[:, 4 * h:5 * h] *= gain
            x = x.to(dt)
            s["k"], s["v"] = x[:, 4 * h:5 * h], x[:, 5 * h:]
        else:
            s["k"] = _keys(gen, (rows, h, d), gain).to(dt)
            s["v"] = torch.randn((rows, h, d), generator=gen, device="cuda").to(dt)
        # what the step changes, read back: new tokens and those that move into the pages
        slot, pos, base, first = [], [], [], 0
        for i in range(slots):
            if step[i] > 0:
                moved = list(range(_cut(before[i], window), _cut(after[i], window)))
                moved = [p for p in moved if p < before[i]] + list(range(before[i], after[i]))
                slot += [i] * len(moved)
                pos += moved
            base.append(first)
            first += max(0, step[i])
        s["read_slot"] = torch.tensor(slot, dtype=torch.int32, device="cuda")
        s["read_pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        if own:
            s["plan"] = kvq.PageTables(state, s["n_new"], rows).run()
            s["call"] = kvq.AppendPages(cache, s["plan"], s["k"], s["v"])
            s["read"] = kvq.PageValues(cache, s["read_slot"], s["read_pos"])
        else:
            grow = [(i, g) for i in range(slots) if step[i] > 0
                    for g in range(_cut(before[i], window) // 32, _cut(after[i], window) // 32)]
            nf = total - used
            for i in range(slots):  # the pages of the step, from the end of the free ones
                for p in range(need[i]):
                    nf -= 1
                    table[i, held[i] + p] = free[nf]
            s["table"] = table.cuda()
            s["groups"] = torch.tensor(grow, dtype=torch.long, device="cuda").view(-1, 2)
            s["base"] = torch.tensor(base, device="cuda")
            s["after"] = torch.tensor(after, device="cuda")
            token = [(i, before[i] + t, base[i] + t) for i in range(slots)
                     for t in range(max(0, step[i]))
                     if before[i] + t >= _cut(after[i], window)]
            s["tail"] = torch.tensor(token, dtype=torch.long, device="cuda").view(-1, 3)
        return s
    if op == "values":
        if case["order"] == "prefix":  # the longest request from its first token on
            i = max(range(slots), key=lambda j: before[j])
            pos = list(range(min(case["rows"], before[i])))
            slot = [i] * len(pos)
        else:
            slot = _host(gen, 0, slots - 1, case["rows"])
            r = torch.rand(case["rows"], generator=gen, device="cuda").tolist()
            pos = [int(x * before[i]) for i, x in zip(slot, r)]
        s["read_slot"] = torch.tensor(slot, dtype=torch.int32, device="cuda")
        s["read_pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        if own:
            s["read"] = kvq.PageValues(cache, s["read_slot"], s["read_pos"])
        return s
    # attend: the last tokens of some requests; rows at the end that stand for none
    each, heads = case["each"], h * case["group"]
    who = torch.randperm(slots, generator=gen, device="cuda").tolist()[:case["rows"] // each]
    slot = [i for i in who for _ in range(each)] + [-1] * case["pad"]
    pos = [before[i] - each + t for i in who for t in range(each)] + [0] * case["pad"]
    s["row_slot"] = torch.tensor(slot, dtype=torch.int32, device="cuda")
    s["row_pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((len(slot), heads, d), generator=gen, device="cuda").bfloat16()
    s["out"] = torch.zeros_like(s["q"])
    if own:
        s["call"] = kvq.AttendPages(cache, s["q"], s["row_slot"],
                                    s["row_pos"] if each > 1 else None, out=s["out"])
    return s


# ------------------------------------------------------------------ plain forms


def _find(inclusive, k):
    """Index of the run that position k of runs laid end to end falls into."""
    return torch.searchsorted(inclusive, k, right=True).clamp(max=inclusive.numel() - 1)


def _plain_tables(s):
    case, dev = s["case"], "cuda"
    window, page, rows, total = case["window"], case["page"], s["rows"], s["total"]
    before, n = s["lengths"].long(), s["n_new"].long()
    grow = n.clamp(min=0)
    held = _pages(before, window, page)
    back = torch.where(n == -1, held, 0)
    after = torch.where(n == -1, 0, before + grow)
    need = (_pages(after, window, page) - held).clamp(min=0)
    back_to, need_to, row_to = back.cumsum(0), need.cumsum(0), grow.cumsum(0)
    n_free = s["n_free"][0].long()
    # the stack of free pages: those given back are put on top, requests take from the top
    k = torch.arange(total, device=dev)
    who = _find(back_to, k)
    page_of = s["table"][who, (k - back_to[who] + back[who]).clamp(0, s["table"].shape[1] - 1)]
    stack = torch.cat((s["free"], s["free"].new_zeros(total + 1)))
    stack[torch.where(k < back_to[-1], n_free + k, 2 * total)] = page_of
    who = _find(need_to, k)
    live = k < need_to[-1]
    column = held[who] + k - need_to[who] + need[who]
    wide = torch.cat((s["table"], s["table"].new_zeros((case["slots"], 1))), 1)
    most = s["table"].shape[1]
    taken = stack[(n_free + back_to[-1] - 1 - k).clamp(min=0)]
    wide[who, torch.where(live, column, most).clamp(0, most)] = taken
    r = torch.arange(rows, device=dev)
    who = _find(row_to, r)
    live = r < row_to[-1]
    position = torch.where(live, before[who] + r - row_to[who] + grow[who], 0)
    offsets = torch.cat((row_to.new_zeros(1), row_to))
    return [wide[:, :most].clone(), offsets.int(), torch.where(live, who, -1).int(),
            position.int(), after.int(), (n_free + back_to[-1] - need_to[-1]).int().view(1)]


def _plain_append(s):
    case, c = s["case"], s["cache"]
    window, page, cap = case["window"], case["page"], _cap(case["window"])
    before = s["lengths"].long()
    slot, g = s["groups"][:, 0], s["groups"][:, 1]
    pos = g[:, None] * 32 + torch.arange(32, device="cuda")
    old = (pos < before[slot][:, None])[:, :, None, None]
    row = (s["base"][slot][:, None] + pos - before[slot][:, None]).clamp(min=0)
    h = torch.arange(case["kv_heads"], device="cuda")
    at = (slot[:, None, None], h, (pos % cap)[:, :, None])
    k = torch.where(old, c["k_ring"][at], s["k"][row]).float()
    v = torch.where(old, c["v_ring"][at], s["v"][row]).float()
    kc, ks = _quantize(k, 1)
    d = case["head_dim"]
    vc, vs = _quantize(v.view(*v.shape[:3], d // 32, 32), 4)
    p = s["table"][slot, g * 32 // page].long()[:, None, None]
    t = (pos % page)[:, :, None]
    c["k_codes"][p, h, t] = kc
    c["v_codes"][p, h, t] = vc.flatten(3)
    c["v_scales"][p, h, t] = vs
    c["k_scales"][p[:, 0], h, (g * 32 % page // 32)[:, None]] = ks
    slot, pos, row = s["tail"].unbind(1)
    c["k_ring"][slot[:, None], h, (pos % cap)[:, None]] = s["k"][row]
    c["v_ring"][slot[:, None], h, (pos % cap)[:, None]] = s["v"][row]
    return _plain_values(s, s["after"])


def _plain_values(s, lengths):
    case, c = s["case"], s["cache"]
    window, page, d = case["window"], case["page"], case["head_dim"]
    slot, pos = s["read_slot"].long(), s["read_pos"].long()
    h = torch.arange(case["kv_heads"], device="cuda")
    p = s["table"][slot, (pos // page).clamp(max=s["table"].shape[1] - 1)].long()
    p, t = p.clamp(min=0)[:, None], (pos % page)[:, None]
    k = c["k_codes"][p, h, t].float() * c["k_scales"][p, h, t // 32]
    v = c["v_codes"][p, h, t].float() * c["v_scales"][p, h, t].repeat_interleave(32, -1)
    packed = (pos < _cut(lengths.long(), window)[slot])[:, None, None]
    r = (pos % _cap(window))[:, None]
    k = torch.where(packed, k, c["k_ring"][slot[:, None], h, r].float())
    v = torch.where(packed, v, c["v_ring"][slot[:, None], h, r].float())
    dt = c["k_ring"].dtype
    return [k.to(dt), v.to(dt)]


def _plain_attend(s):
    case, c, q = s["case"], s["cache"], s["q"]
    window, page, cap, d = case["window"], case["page"], _cap(case["window"]), case["head_dim"]
    hk, rows = case["kv_heads"], q.shape[0]
    slot = s["row_slot"].long().clamp(min=0)
    last = s["row_pos"].long()
    cut = _cut(s["lengths"].long(), window)[slot]
    p = s["table"][slot].long().clamp(min=0)  # [rows][pages]
    tokens = p.shape[1] * page
    kc = c["k_codes"][p].transpose(1, 2).reshape(rows, hk, tokens, d)
    ks = c["k_scales"][p].transpose(1, 2).reshape(rows, hk, tokens // 32, 1, d)
    k = torch.cat(((kc.view(rows, hk, -1, 32, d) * ks).flatten(2, 3),
                   c["k_ring"][slot].float()), 2)
    x = q.float().view(rows, hk, -1, d)
    a = (x @ k.transpose(2, 3)) * (d ** -0.5)
    del kc, k
    at = torch.arange(tokens, device="cuda")
    w = torch.arange(cap, device="cuda")
    w = cut[:, None] + (w - cut[:, None]) % cap
    seen = torch.cat(((at < cut[:, None]) & (at <= last[:, None]), w <= last[:, None]), 1)
    a = a.masked_fill_(~seen[:, None, None], float("-inf"))
    a = (a - a.amax(-1, keepdim=True)).exp_()
    a = a / a.sum(-1, keepdim=True)
    vc = c["v_codes"][p].transpose(1, 2).reshape(rows, hk, tokens, d // 32, 32)
    vs = c["v_scales"][p].transpose(1, 2).reshape(rows, hk, tokens, d // 32, 1)
    v = torch.cat(((vc * vs).flatten(3), c["v_ring"][slot].float()), 2)
    o = (a @ v).view(rows, -1, d).to(q.dtype)
    return torch.where((s["row_slot"] >= 0)[:, None, None], o, s["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "tables":
            plan = state["call"].run(advance=False)
            return [plan.state.table, plan.offsets, plan.row_slot, plan.positions, plan.after,
                    plan.free_after]
        if op == "append":
            state["call"].run()
            return state["read"].run()
        if op == "values":
            return state["read"].run()
        return state["call"].run()
    if op == "tables":
        return _plain_tables(state)
    if op == "append":
        return _plain_append(state)
    if op == "values":
        return _plain_values(state, state["lengths"])
    return _plain_attend(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    """Of the mean over the inputs that `prepare` makes: lengths are uniform over their range."""
    op, window, page, slots = case["op"], case["window"], case["page"], case["slots"]
    if op in ("tables", "append"):
        mean = 0.75 * case["prompt"] * case["prompts"]
        single = max(0, slots - case["prompts"] - case["idle"] - case.get("leave", 0))
        rows = mean + single
    if op == "tables":
        new = max(0.0, mean - case["prompts"] * window) / page
        left = case["leave"] * max(0.0, case["longest"] / 2 - window) / page
        return {"bytes": 8 * slots + 8 * _rows(case) + 8 * slots + 8 * (new + left), "flops": 0}
    d, h = case["head_dim"], case["kv_heads"]
    el = 4 if case.get("dtype") == "f32" else 2
    if op == "append":
        # a decoding request completes a group of 32 tokens every 32nd step: one token a step
        moved = single if case["longest"] > window else 0
        tail = single + case["prompts"] * min(window + 16, 0.75 * case["prompt"])
        packed = rows - tail + moved
        changed = 1.25 * d * packed + 2 * d * el * tail  # written, and read back
        return {"bytes": h * (2 * d * el * (rows + moved) + 2 * changed
                              + 2 * d * el * (rows + moved)), "flops": 0}
    if op == "values":
        rows = min(case["rows"], case["longest"]) if case["order"] == "prefix" else case["rows"]
        return {"bytes": h * rows * (1.25 * d + 2 * d * el) + 8 * rows, "flops": 0}
    length = (case["shortest"] + case["longest"]) / 2
    float_rows = min(window + 16, length)
    asked = case["rows"] // case["each"]
    cache = asked * h * (1.25 * d * (length - float_rows) + 4 * d * float_rows)
    heads = h * case["group"]
    return {"bytes": cache + case["rows"] * heads * d * 4 + 4 * case["rows"],
            "flops": 4.0 * case["rows"] * heads * d * length}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_tables(s):
    """The tables step by step, on the host."""
    case = s["case"]
    window, page = case["window"], case["page"]
    table, free = s["table"].tolist(), s["free"].tolist()
    before, step = s["lengths"].tolist(), s["n_new"].tolist()
    free = free[:int(s["n_free"][0])]
    for i, n in enumerate(step):
        if n == -1:
            free += table[i][:_pages(before[i], window, page)]
    offsets, slot, pos, after = [0], [], [], []
    for i, n in enumerate(step):
        if n == -1:
            after.append(0)
        else:
            for p in range(_pages(before[i], window, page), _pages(before[i] + n, window, page)):
                table[i][p] = free.pop()
            slot += [i] * n
            pos += range(before[i], before[i] + n)
            after.append(before[i] + n)
        offsets.append(len(slot))
    rest = s["rows"] - len(slot)
    out = [table, offsets, slot + [-1] * rest, pos + [0] * rest, after, [len(free)]]
    return [torch.tensor(x, dtype=torch.int64, device="cuda") for x in out]


def _round32(x):
    return x.float().double()


def _group64(x):
    """The values that int4 leaves of groups along the last axis."""
    top = x.abs().amax(-1, keepdim=True)
    scale = _round32(top / torch.full_like(top, 7.0))
    unit = torch.where(scale > 0, scale, torch.ones_like(scale))
    return _round32(x / unit).round().clamp(-7, 7) * scale


def _token64(s, i, length):
    """Keys and values of the request in slot i, [heads][length][d], as the cache holds them."""
    case, c = s["case"], s["cache"]
    cut, page, cap = _cut(length, case["window"]), case["page"], _cap(case["window"])
    p = s["table"][i, :-(-cut // page)].long()
    h, d = case["kv_heads"], case["head_dim"]
    k = c["k_codes"][p].double().view(-1, h, page // 32, 32, d)
    k = (k * c["k_scales"][p].double()[:, :, :, None]).transpose(0, 1).reshape(h, -1, d)[:, :cut]
    v = c["v_codes"][p].double().view(-1, h, page, d // 32, 32)
    v = (v * c["v_scales"][p].double()[..., None]).transpose(0, 1).reshape(h, -1, d)[:, :cut]
    w = [t % cap for t in range(cut, length)]
    return (torch.cat((k, c["k_ring"][i][:, w].double()), 1),
            torch.cat((v, c["v_ring"][i][:, w].double()), 1))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "tables":
        return _exact_tables(s)
    h, d = case["kv_heads"], case["head_dim"]
    before = s["lengths"].tolist()
    if op in ("append", "values"):
        slot, pos = s["read_slot"].long(), s["read_pos"].long()
        k = torch.zeros((slot.numel(), h, d), dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        step = s["n_new"].tolist()
        first = 0
        for i in range(case["slots"]):
            n = max(0, step[i]) if op == "append" else 0
            mine = (slot == i).nonzero().flatten()
            if mine.numel():
                ki, vi = _token64(s, i, before[i])
                if n:
                    ki = torch.cat((ki, s["k"][first:first + n].double().transpose(0, 1)), 1)
                    vi = torch.cat((vi, s["v"][first:first + n].double().transpose(0, 1)), 1)
                    lo, hi = _cut(before[i], case["window"]), _cut(before[i] + n, case["window"])
                    if hi > lo:
                        x = ki[:, lo:hi].reshape(h, -1, 32, d).transpose(2, 3)
                        ki[:, lo:hi] = _group64(x).transpose(2, 3).reshape(h, -1, d)
                        x = vi[:, lo:hi].reshape(h, hi - lo, d // 32, 32)
                        vi[:, lo:hi] = _group64(x).reshape(h, -1, d)
                k[mine], v[mine] = (x[:, pos[mine]].transpose(0, 1) for x in (ki, vi))
            first += n
        return [k, v]
    if 4.0 * case["rows"] * h * case["group"] * d * case["longest"] > 6e11:
        return None
    out = s["out"].double()
    q = s["q"].double()
    for r, (i, p) in enumerate(zip(s["row_slot"].tolist(), s["row_pos"].tolist())):
        if i < 0:
            continue
        k, v = _token64(s, i, before[i])
        for j in range(h):
            x = q[r, j * case["group"]:(j + 1) * case["group"]]
            a = (x @ k[j, :p + 1].T) / math.sqrt(d)
            out[r, j * case["group"]:(j + 1) * case["group"]] = torch.softmax(a, 1) @ v[j, :p + 1]
    return out
