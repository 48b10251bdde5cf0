"""Rotary positions, tree attention and block-sparse attention over the packed
KV cache: the cases they are timed on, their inputs and their plain forms.

``run`` computes an operator with elementary torch operations in fp32 while
``own`` is false, and with the library's calls when it is true; ``exact``
computes the same outputs from the definitions in fp64.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decoding step of a full batch: q and k rows of the projection, far positions
        dict(name="rope_decode_b64", op="rope", batch=64, n=1, q_heads=16, kv_heads=2,
             head_dim=128, rotary=128, layout="half", scaling="none", dtype="bf16",
             rows=True, inverse=False, far=32768),
        # the prompt of a long-context request, read from the projection's rows
        dict(name="rope_prompt_scaled", op="rope", batch=2, n=8192, q_heads=16, kv_heads=2,
             head_dim=128, rotary=128, layout="half", scaling="ramp", dtype="bf16",
             rows=True, inverse=False, far=131072),
        # the rotation taken back (its gradient), interleaved pairs, half of the head, fp32
        dict(name="rope_inverse_partial_f32", op="rope", batch=3, n=1023, q_heads=16, kv_heads=2,
             head_dim=128, rotary=64, layout="interleaved", scaling="bands", dtype="f32",
             rows=False, inverse=True, far=65536),
        # one request checking a single drafted token: latency
        dict(name="tree_b1_t1", op="tree", batch=1, tokens=1, n=1024, recent=128, kv_heads=2,
             group=8, shape="chain", pad=False),
        # a short draft of a medium batch, sequences with smaller trees padded
        dict(name="tree_b16_t8_pad", op="tree", batch=16, tokens=8, n=8200, recent=136,
             kv_heads=2, group=8, shape="tree", pad=True),
        # an odd tree over a large batch of medium contexts
        dict(name="tree_b64_t21", op="tree", batch=64, tokens=21, n=8191, recent=159,
             kv_heads=2, group=8, shape="tree", pad=False),
        # a wide draft tree over long contexts
        dict(name="tree_b16_t64_32k", op="tree", batch=16, tokens=64, n=32768, recent=128,
             kv_heads=2, group=8, shape="tree", pad=False),
        # block summaries of a long cache, once after its prompt
        dict(name="summary_b32_128k", op="summary", batch=32, n=131072, recent=128, kv_heads=2,
             head_dim=128, block=64, new=0),
        # ... and of the blocks that the last appends completed
        dict(name="summary_step_b64", op="summary", batch=64, n=8192, recent=128, kv_heads=2,
             head_dim=128, block=64, new=2),
        # block-sparse decoding of one request: latency
        dict(name="sparse_b1_32k", op="sparse", batch=1, queries=1, n=32768, recent=128,
             kv_heads=2, group=8, block=64, top_k=16, sink=1),
        # block-sparse decoding of a batch of very long contexts
        dict(name="sparse_b32_128k", op="sparse", batch=32, queries=1, n=131072, recent=128,
             kv_heads=2, group=8, block=64, top_k=32, sink=1),
        # several query tokens a sequence, each with its own blocks, odd sizes
        dict(name="sparse_b16_q5", op="sparse", batch=16, queries=5, n=8213, recent=149,
             kv_heads=2, group=8, block=32, top_k=25, sink=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "summary", "sparse", "sparse"])
    if op == "rope":
        d = rng.choice([64, 128, 128, 256])
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, n=max(1, min(_log(rng, 1, 8192), 8192 // batch)),
                    q_heads=rng.choice([8, 16, 32]), kv_heads=rng.choice([1, 2, 8]), head_dim=d,
                    rotary=rng.choice([d, d, d // 2]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "ramp", "bands"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, far=_log(rng, 4096, 1 << 20))
    batch = _log(rng, 1, 64)
    if op == "tree":
        kv_heads, group = rng.choice([(2, 8), (2, 8), (4, 4), (1, 7), (2, 5)])
        n = _log(rng, 130, 32768)
        tokens = _log(rng, 1, 64)
        while batch * n > 16 * 32768:
            batch -= 1
        return dict(op=op, batch=batch, tokens=tokens, n=n, recent=rng.randint(0, 129),
                    kv_heads=kv_heads, group=group, shape=rng.choice(["tree", "chain"]),
                    pad=rng.random() < 0.4)
    if op == "summary":
        n = _log(rng, 200, 131072)
        while batch * n > 32 * 131072:
            batch -= 1
        return dict(op=op, batch=batch, n=n, recent=rng.randint(0, 160), kv_heads=2,
                    head_dim=rng.choice([64, 128, 128, 256]) if n < 40000 else 128,
                    block=rng.choice([32, 64, 128]), new=rng.choice([0, 0, 1, 3]))
    kv_heads, group = rng.choice([(2, 8), (2, 8), (4, 4), (1, 7)])
    queries = rng.choice([1, 1, 1, rng.randint(2, 6)])
    n = _log(rng, 200, 131072)
    while batch * n > 32 * 131072 or batch * queries > 80:
        batch -= 1
    return dict(op=op, batch=batch, queries=queries, n=n, recent=rng.randint(0, 160),
                kv_heads=kv_heads, group=group, block=rng.choice([32, 64, 128]),
                top_k=_log(rng, 4, 32), sink=rng.randint(0, 2))


# ------------------------------------------------------------------ inputs


def _quantize_k(k, cut):
    """Grouped int4 of the first `cut` tokens: one scale per (32-token group, channel)."""
    b, h, _, d = k.shape
    gk = -(-cut // 32)
    x = torch.zeros((b, h, gk * 32, d), dtype=torch.float32, device=k.device)
    x[:, :, :cut] = k[:, :, :cut]
    x = x.view(b, h, gk, 32, d)
    scale = x.abs().amax(3) / 7.0
    code = torch.where(scale.unsqueeze(3) > 0, torch.round(x / scale.unsqueeze(3)),
                       torch.zeros_like(x)).clamp_(-7, 7).to(torch.int8)
    return code, scale


def _quantize_v(v, cut):
    b, h, _, d = v.shape
    x = v[:, :, :cut].float().reshape(b, h, cut, d // 32, 32)
    scale = x.abs().amax(4) / 7.0
    code = torch.where(scale.unsqueeze(4) > 0, torch.round(x / scale.unsqueeze(4)),
                       torch.zeros_like(x)).clamp_(-7, 7).to(torch.int8)
    return code.view(b, h, cut, d), scale


def _nibbles(code):
    u = (code + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _make_cache(batch, kv_heads, n, d, recent, gen):
    """Packed arrays of a cache: keys with a few strong channels, as trained keys have them."""
    dev = "cuda"
    cut = n - recent
    gain = 0.5 + torch.rand((1, kv_heads, 1, d), generator=gen, device=dev)
    gain = gain * torch.where(torch.rand((1, kv_heads, 1, d), generator=gen, device=dev) < 0.03,
                              4.0, 1.0)
    gk = -(-cut // 32)
    c = dict(batch=batch, kv_heads=kv_heads, n=n, d=d, recent=recent, cut=cut, gk=gk)
    c["k_codes"] = torch.empty((batch, kv_heads, gk, 32, d // 2), dtype=torch.uint8, device=dev)
    c["k_scales"] = torch.empty((batch, kv_heads, gk, d), device=dev)
    c["v_codes"] = torch.empty((batch, kv_heads, cut, d // 2), dtype=torch.uint8, device=dev)
    c["v_scales"] = torch.empty((batch, kv_heads, cut, d // 32), device=dev)
    c["k_window"] = torch.empty((batch, kv_heads, recent, d), dtype=torch.bfloat16, device=dev)
    c["v_window"] = torch.empty((batch, kv_heads, recent, d), dtype=torch.bfloat16, device=dev)
    step = max(1, (1 << 27) // (kv_heads * n * d))  # sequences made at a time
    for b0 in range(0, batch, step):
        nb = min(step, batch - b0)
        k = torch.randn((nb, kv_heads, n, d), generator=gen, device=dev).mul_(gain).bfloat16()
        v = torch.randn((nb, kv_heads, n, d), generator=gen, device=dev).bfloat16()
        sl = slice(b0, b0 + nb)
        if cut:
            code, scale = _quantize_k(k, cut)
            c["k_codes"][sl], c["k_scales"][sl] = _nibbles(code), scale
            code, scale = _quantize_v(v, cut)
            c["v_codes"][sl], c["v_scales"][sl] = _nibbles(code), scale
        c["k_window"][sl], c["v_window"][sl] = k[:, :, cut:], v[:, :, cut:]
    return c


def _own_cache(c):
    """The library's cache with the same contents, laid out with room for appends."""
    from quantized_sparse_kv_gb300 import kvq
    cache = kvq.PackedCache(c["batch"], c["kv_heads"], c["n"], c["d"], c["recent"], "bf16",
                            "bf16", reserve=(c["gk"] + 4, c["recent"] + 64))
    for name, view in cache.used().items():
        view.copy_(c[name])
    return cache


def _parents(batch, tokens, shape, pad, gen):
    """Parent of every drafted token (-1: the cache's last token, -2: no token)."""
    r = torch.rand((batch, tokens), generator=gen, device="cuda").cpu()
    out = torch.empty((batch, tokens), dtype=torch.int32)
    for b in range(batch):
        for i in range(tokens):
            out[b, i] = i - 1 if shape == "chain" or i == 0 else int(r[b, i] * (i + 1)) - 1
        if pad and b % 2:
            out[b, tokens - int(r[b, 0] * tokens):] = -2
    return out.cuda()


def _ancestors(parents):
    """seen[b, i, j]: drafted token i sees drafted token j (itself and its ancestors)."""
    p = parents.cpu()
    batch, t = p.shape
    seen = torch.zeros((batch, t, t), dtype=torch.bool)
    for b in range(batch):
        for i in range(t):
            if p[b, i] >= 0:
                seen[b, i] = seen[b, int(p[b, i])]
            if p[b, i] > -2:
                seen[b, i, i] = True
    return seen.to(parents.device)


_SCALING = {
    "none": dict(), "linear": dict(factor=4.0), "base": dict(factor=4.0),
    "ramp": dict(factor=8.0, original=16384, fast=32.0, slow=1.0),
    "bands": dict(factor=8.0, original=8192, low=1.0, high=4.0),
}


def _frequencies(rotary, scaling, base=10000.0):
    """Angular frequency of every pair and the amplitude of the rotation, in 64 bits."""
    s, half = _SCALING[scaling], rotary // 2
    if scaling == "base":
        base = base * s["factor"] ** (rotary / (rotary - 2.0))
    f = [base ** (-2.0 * i / rotary) for i in range(half)]
    if scaling == "linear":
        return [x / s["factor"] for x in f], 1.0
    if scaling == "ramp":
        def index(turns):
            return rotary * math.log(s["original"] / (2.0 * math.pi * turns)) / (2.0 * math.log(base))
        lo = max(0.0, float(math.floor(index(s["fast"]))))
        hi = min(rotary - 1.0, float(math.ceil(index(s["slow"]))))
        if hi == lo:
            hi += 0.001
        out = []
        for i, x in enumerate(f):
            w = min(1.0, max(0.0, (i - lo) / (hi - lo)))
            out.append(x / s["factor"] * w + x * (1.0 - w))
        return out, 0.1 * math.log(s["factor"]) + 1.0
    if scaling == "bands":
        out = []
        for x in f:
            turns = s["original"] * x / (2.0 * math.pi)
            w = min(1.0, max(0.0, (turns - s["low"]) / (s["high"] - s["low"])))
            out.append(x / s["factor"] * (1.0 - w) + x * w)
        return out, 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "rope":
        b, n, d = case["batch"], case["n"], case["head_dim"]
        hq, hk = case["q_heads"], case["kv_heads"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["rows"]:  # one row per token: q heads, k heads, v heads
            x = torch.randn((b, n, hq + 2 * hk, d), generator=gen, device="cuda").to(dt)
            s["q"] = x[:, :, :hq].transpose(1, 2)
            s["k"] = x[:, :, hq:hq + hk].transpose(1, 2)
        else:
            s["q"] = torch.randn((b, hq, n, d), generator=gen, device="cuda").to(dt)
            s["k"] = torch.randn((b, hk, n, d), generator=gen, device="cuda").to(dt)
        start = torch.randint(0, max(1, case["far"] - n), (b, 1), generator=gen, device="cuda")
        s["pos"] = (start + torch.arange(n, device="cuda")).to(torch.int32)
        if own:
            from quantized_sparse_kv_gb300 import kvq
            plan = kvq.RopePlan(case["rotary"], layout=case["layout"], scaling=case["scaling"],
                                **_SCALING[case["scaling"]])
            s["call"] = kvq.Rope(plan, s["q"], s["k"], s["pos"], inverse=case["inverse"])
        else:
            f, s["amp"] = _frequencies(case["rotary"], case["scaling"])
            s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        return s
    d = case.get("head_dim", 128)
    c = _make_cache(case["batch"], case["kv_heads"], case["n"], d, min(case["recent"], case["n"]),
                    gen)
    if op == "summary":
        s["block"] = case["block"]
        blocks = -(-c["cut"] // case["block"])
        s["first"] = max(0, blocks - case["new"]) if case["new"] else 0
        if own:
            from quantized_sparse_kv_gb300 import kvq
            s["cache"] = _own_cache(c)
            s["call"] = kvq.BlockSummary(s["cache"], case["block"])
        else:
            s["cache"] = c
        return s
    heads = case["kv_heads"] * case["group"]
    if op == "tree":
        b, t = case["batch"], case["tokens"]
        q = torch.randn((b, heads, t, 128), generator=gen, device="cuda").bfloat16()
        k = torch.randn((b, case["kv_heads"], t, 128), generator=gen, device="cuda").bfloat16()
        v = torch.randn((b, case["kv_heads"], t, 128), generator=gen, device="cuda").bfloat16()
        par = _parents(b, t, case["shape"], case["pad"], gen)
        out = torch.zeros((b, heads, t, 128), dtype=torch.bfloat16, device="cuda")
        if own:
            from quantized_sparse_kv_gb300 import kvq
            s["cache"] = _own_cache(c)
            s["call"] = kvq.AttendTree(s["cache"], q, k, v, par, out=out)
        else:
            s.update(cache=c, q=q, k=k, v=v, parents=par, out=out)
        return s
    nq = case["queries"]
    q = torch.randn((case["batch"], heads, nq, 128), generator=gen, device="cuda").bfloat16()
    if own:
        from quantized_sparse_kv_gb300 import kvq
        s["cache"] = _own_cache(c)
        s["summary"] = kvq.BlockSummary(s["cache"], case["block"])
        s["summary"].update()
        s["call"] = kvq.AttendBlocks(s["cache"], q, s["summary"], case["top_k"],
                                     n_sink=case["sink"])
    else:
        codes, scales = _plain_summary(c, case["block"], 0)
        s.update(cache=c, q=q, sum_codes=codes.to(torch.int8), sum_scales=scales)
    return s


# ------------------------------------------------------------------ plain forms


def _codes(u8):
    """int4 codes as fp32, the last axis doubled."""
    lo = (u8 & 15).float() - 8.0
    hi = (u8 >> 4).float() - 8.0
    return torch.stack((lo, hi), -1).flatten(-2)


def _keys(c, b0, b1):
    k = _codes(c["k_codes"][b0:b1]) * c["k_scales"][b0:b1].unsqueeze(3)
    k = k.flatten(2, 3)[:, :, :c["cut"]]
    return torch.cat((k, c["k_window"][b0:b1].float()), 2)


def _values(c, b0, b1):
    v = _codes(c["v_codes"][b0:b1]) * c["v_scales"][b0:b1].repeat_interleave(32, -1)
    return torch.cat((v, c["v_window"][b0:b1].float()), 2)


def _plain_rope(s):
    case = s["case"]
    r = case["rotary"]
    ang = s["pos"].double().unsqueeze(-1) * s["freq"]
    cos = (ang.cos() * s["amp"]).float().unsqueeze(1)
    sin = (ang.sin() * s["amp"]).float().unsqueeze(1)
    if case["inverse"]:
        sin = -sin
    outs = []
    for x in (s["q"], s["k"]):
        y = x.float()
        rot, rest = y[..., :r], y[..., r:]
        if case["layout"] == "half":
            a, b = rot[..., :r // 2], rot[..., r // 2:]
            rot = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        outs.append(torch.cat((rot, rest), -1).to(x.dtype))
    return outs


def _plain_tree(s):
    c, q = s["cache"], s["q"]
    batch, heads, t, d = q.shape
    hk = c["kv_heads"]
    g = heads // hk
    seen = _seen_plain(s["parents"])
    out = s["out"].clone()
    step = max(1, (1 << 31) // (heads * t * (c["n"] + t)))
    for b0 in range(0, batch, step):
        b1 = min(batch, b0 + step)
        k = torch.cat((_keys(c, b0, b1), s["k"][b0:b1].float()), 2)
        v = torch.cat((_values(c, b0, b1), s["v"][b0:b1].float()), 2)
        x = q[b0:b1].float().reshape(b1 - b0, hk, g * t, d)
        p = (x @ k.transpose(2, 3)).view(b1 - b0, hk, g, t, -1) * (d ** -0.5)
        p[..., c["n"]:].masked_fill_(~seen[b0:b1, None, None], float("-inf"))
        p = (p - p.amax(-1, keepdim=True)).exp_()
        p = p / p.sum(-1, keepdim=True)
        o = (p.view(b1 - b0, hk, g * t, -1) @ v).view(b1 - b0, heads, t, d)
        keep = (s["parents"][b0:b1] > -2)[:, None, :, None]
        out[b0:b1] = torch.where(keep, o.to(out.dtype), out[b0:b1])
    return out


def _seen_plain(parents):
    """Ancestor mask on the device: the parent relation closed by squaring."""
    t = parents.shape[1]
    at = torch.arange(t, device=parents.device)
    step = (parents.unsqueeze(2) == at) | (at.unsqueeze(1) == at)
    seen = (step & (parents > -2).unsqueeze(2)).float()
    hops = 1
    while hops < t:
        seen = (seen @ seen > 0).float()
        hops *= 2
    return seen > 0


def _over_127(x):
    """x / 127, correctly rounded (a division by a number would multiply by its reciprocal)."""
    return x / torch.full_like(x, 127.0)


def _plain_summary(c, block, first):
    m = block // 32
    blocks = -(-c["cut"] // block)
    g0 = first * m
    b, h, d = c["batch"], c["kv_heads"], c["d"]
    total = torch.zeros((b, h, (blocks - first) * m, d), device=c["k_codes"].device)
    step = max(1, (1 << 29) // (h * (c["gk"] - g0 + 1) * 32 * d))
    for b0 in range(0, b, step):
        part = _codes(c["k_codes"][b0:b0 + step, :, g0:]).sum(3)
        total[b0:b0 + step, :, :c["gk"] - g0] = part * c["k_scales"][b0:b0 + step, :, g0:]
    total = total.view(b, h, blocks - first, m, d)
    acc = total[:, :, :, 0]
    for i in range(1, m):
        acc = acc + total[:, :, :, i]
    count = torch.full((blocks,), float(block), device=acc.device)
    if blocks:
        count[-1] = c["cut"] - block * (blocks - 1)
    mean = acc / count[first:, None]
    scale = _over_127(mean.abs().amax(-1))
    code = torch.where(scale.unsqueeze(-1) > 0, torch.round(mean / scale.unsqueeze(-1)),
                       torch.zeros_like(mean))
    return code, scale


def _plain_select(q, codes, scales, kv_heads, top_k, sink):
    """[batch][kv_heads][queries][top_k] blocks, ascending, -1 behind the last."""
    batch, heads, nq, d = q.shape
    x = q.float().view(batch, kv_heads, heads // kv_heads * nq, d)
    sq = _over_127(x.abs().amax(-1))
    qi = torch.where(sq.unsqueeze(-1) > 0, torch.round(x / sq.unsqueeze(-1)),
                     torch.zeros_like(x))
    dot = qi @ codes.float().transpose(2, 3)
    score = (sq.unsqueeze(-1) * scales.unsqueeze(2)) * dot
    score = score.view(batch, kv_heads, heads // kv_heads, nq, -1).amax(2)
    score[..., :sink] = float("inf")
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top_k]
    picked = order.sort(-1).values.int()
    if picked.shape[-1] < top_k:
        tail = picked.new_full((*picked.shape[:-1], top_k - picked.shape[-1]), -1)
        picked = torch.cat((picked, tail), -1)
    return picked


def _plain_sparse(s):
    c, q, case = s["cache"], s["q"], s["case"]
    batch, heads, nq, d = q.shape
    hk, block = c["kv_heads"], case["block"]
    g = heads // hk
    picked = _plain_select(q, s["sum_codes"], s["sum_scales"], hk, case["top_k"], case["sink"])
    tok = picked.long().unsqueeze(-1) * block + torch.arange(block, device=q.device)
    ok = (picked.unsqueeze(-1) >= 0) & (tok < c["cut"])
    tok = torch.where(ok, tok, torch.zeros_like(tok)).flatten(-2)  # [b][hk][nq][L]
    ok = ok.flatten(-2)
    bi = torch.arange(batch, device=q.device).view(-1, 1, 1, 1)
    hi = torch.arange(hk, device=q.device).view(1, -1, 1, 1)
    parts_k, parts_v = [], []
    if c["cut"]:
        kc = c["k_codes"].flatten(2, 3)
        parts_k.append(_codes(kc[bi, hi, tok]) * c["k_scales"][bi, hi, tok // 32])
        parts_v.append(_codes(c["v_codes"][bi, hi, tok])
                       * c["v_scales"][bi, hi, tok].repeat_interleave(32, -1))
    else:
        ok = ok[..., :0]
    win = (batch, hk, nq, c["recent"], d)
    parts_k.append(c["k_window"].float().unsqueeze(2).expand(win))
    parts_v.append(c["v_window"].float().unsqueeze(2).expand(win))
    k, v = torch.cat(parts_k, 3), torch.cat(parts_v, 3)
    x = q.float().view(batch, hk, g, nq, d).transpose(2, 3)
    p = (x @ k.transpose(3, 4)) * (d ** -0.5)
    seen = torch.cat((ok, ok.new_ones((batch, hk, nq, c["recent"]))), -1)
    p = p.masked_fill(~seen.unsqueeze(3), float("-inf"))
    p = (p - p.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    o = (p @ v).transpose(2, 3).reshape(batch, heads, nq, d)
    return [o.to(q.dtype), picked]


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "summary":
            state["call"].update(first=state["first"])
            return state["call"].values(state["first"])
        if op == "sparse":
            out = state["call"].run()
            return [out, state["call"].selected]
        return state["call"].run()
    if op == "rope":
        return _plain_rope(state)
    if op == "tree":
        return _plain_tree(state)
    if op == "summary":
        code, scale = _plain_summary(state["cache"], state["block"], state["first"])
        return code * scale.unsqueeze(-1)
    return _plain_sparse(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op, b = case["op"], case["batch"]
    if op == "rope":
        el = 2 if case["dtype"] == "bf16" else 4
        vals = b * case["n"] * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
        rot = b * case["n"] * (case["q_heads"] + case["kv_heads"]) * case["rotary"]
        return {"bytes": 2 * vals * el + 4 * b * case["n"] + 4 * case["rotary"], "flops": 3 * rot}
    d = case.get("head_dim", 128)
    recent = min(case["recent"], case["n"])
    cut = case["n"] - recent
    units = b * case["kv_heads"]
    gk = -(-cut // 32)
    if op == "tree":
        t, hq = case["tokens"], case["kv_heads"] * case["group"]
        cache = units * (gk * (16 * d + 4 * d) + cut * (d // 2 + d // 8) + recent * 4 * d)
        rows = b * t * (2 * hq + 2 * case["kv_heads"]) * d * 2
        flops = 4 * b * hq * t * d * (case["n"] + (t + 1) / 2)
        return {"bytes": cache + rows + 4 * b * t, "flops": flops}
    blocks = -(-cut // case["block"])
    if op == "summary":
        nb = min(blocks, case["new"]) if case["new"] else blocks
        groups = min(gk, nb * (case["block"] // 32))
        return {"bytes": units * (groups * 20 * d + nb * 4 * d), "flops": units * groups * 32 * d}
    nq, hq = case["queries"], case["kv_heads"] * case["group"]
    top = min(case["top_k"], blocks)
    tokens = min(cut, top * case["block"])
    distinct = min(cut, nq * tokens)  # several queries may choose the same blocks
    distinct = max(tokens, distinct // max(1, nq))
    data = (units * blocks * (d + 4) + units * distinct * (d // 2 + d // 8)
            + units * distinct * (d // 2 + 4 * d // 32) + units * recent * 4 * d)
    rows = 2 * b * hq * nq * d * 2 + 4 * units * nq * case["top_k"]
    flops = 2 * b * hq * nq * d * blocks + 4 * b * hq * nq * d * (tokens + recent)
    return {"bytes": data + rows, "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits


def _unpack64(u8):
    n = u8.to(torch.int16)
    out = torch.empty((*u8.shape[:-1], u8.shape[-1] * 2), dtype=torch.float64, device=u8.device)
    out[..., 0::2] = ((n & 15) - 8).double()
    out[..., 1::2] = ((n >> 4) - 8).double()
    return out


def _cache64(c, b, h):
    """Keys and values of one (sequence, KV head) as attention reads them."""
    k = _unpack64(c["k_codes"][b, h]) * c["k_scales"][b, h].double()[:, None]
    k = torch.cat((k.reshape(-1, c["d"])[:c["cut"]], c["k_window"][b, h].double()))
    v = _unpack64(c["v_codes"][b, h]).view(c["cut"], c["d"] // 32, 32)
    v = (v * c["v_scales"][b, h].double()[..., None]).reshape(c["cut"], c["d"])
    return k, torch.cat((v, c["v_window"][b, h].double()))


def _round32(x):
    return x.float().double()


def _summary64(c, block):
    """Codes and scales by the definition: every named step rounded once to fp32."""
    m = block // 32
    codes, scales = [], []
    for b in range(c["batch"]):
        for h in range(c["kv_heads"]):
            sums = _unpack64(c["k_codes"][b, h]).sum(1)
            part = _round32(sums * c["k_scales"][b, h].double())
            uc, us = [], []
            blocks = -(-c["cut"] // block)
            pad = torch.zeros((blocks * m - c["gk"], c["d"]), dtype=torch.float64,
                              device=part.device)
            part = torch.cat((part, pad)).view(blocks, m, c["d"])
            acc = part[:, 0]
            for i in range(1, m):
                acc = _round32(acc + part[:, i])
            tokens = (c["cut"] - block * torch.arange(blocks, device=part.device)).clamp(max=block)
            mean = _round32(acc / tokens.double()[:, None])
            s = _round32(mean.abs().amax(1) / 127.0) if blocks else acc.new_zeros(0)
            q = _round32(mean / torch.where(s > 0, s, torch.ones_like(s))[:, None]).round()
            uc.append(torch.where((s > 0)[:, None], q, torch.zeros_like(q)))
            us.append(s)
            codes.append(uc[0])
            scales.append(us[0])
    shape = (c["batch"], c["kv_heads"], -1)
    return torch.stack(codes).view(*shape, c["d"]) if codes[0].numel() else None, \
        torch.stack(scales).view(*shape)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rope":
        f, amp = _frequencies(case["rotary"], case["scaling"])
        half = case["rotary"] // 2
        turn = torch.polar(torch.full((half,), amp, dtype=torch.float64, device="cuda"),
                           torch.zeros(half, dtype=torch.float64, device="cuda"))
        ang = s["pos"].double()[:, None, :, None] * torch.tensor(f, dtype=torch.float64,
                                                                 device="cuda")
        turn = turn * torch.polar(torch.ones_like(ang), -ang if case["inverse"] else ang)
        outs = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            if case["layout"] == "half":
                i0, i1 = slice(0, half), slice(half, 2 * half)
            else:
                i0, i1 = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
            z = torch.complex(y[..., i0], y[..., i1]) * turn
            y[..., i0], y[..., i1] = z.real, z.imag
            outs.append(y)
        return outs
    c = s["cache"]
    if op == "summary":
        codes, scales = _summary64(c, case["block"])
        return _round32(codes * scales[..., None])[:, :, s["first"]:]
    group, hk = case["group"], case["kv_heads"]
    q = s["q"].double()
    out = torch.empty_like(q)
    if op == "tree":
        n, t = case["n"], case["tokens"]
        if 4.0 * case["batch"] * q.shape[1] * t * n * 128 > 6e11:
            return None
        seen = _ancestors(s["parents"])
        for b in range(case["batch"]):
            for h in range(hk):
                k, v = _cache64(c, b, h)
                k = torch.cat((k, s["k"][b, h].double()))
                v = torch.cat((v, s["v"][b, h].double()))
                for j in range(h * group, (h + 1) * group):
                    a = (q[b, j] @ k.T) / math.sqrt(128.0)
                    a[:, n:][~seen[b]] = -math.inf
                    out[b, j] = torch.softmax(a, 1) @ v
        return torch.where((s["parents"] == -2)[:, None, :, None], s["out"].double(), out)
    codes, scales = _summary64(c, case["block"])
    blocks = scales.shape[-1]
    nq, top = case["queries"], case["top_k"]
    picked = torch.full((case["batch"], hk, nq, top), -1, dtype=torch.int32, device="cuda")
    for b in range(case["batch"]):
        for h in range(hk):
            k, v = _cache64(c, b, h)
            for i in range(nq):
                x = q[b, h * group:(h + 1) * group, i]
                chosen = []
                if blocks:
                    sx = _round32(x.abs().amax(1) / 127.0)
                    xi = _round32(x / torch.where(sx > 0, sx, torch.ones_like(sx))[:, None]).round()
                    xi = xi * (sx > 0)[:, None]
                    w = _round32(sx[:, None] * scales[b, h][None])
                    best = _round32(w * (xi @ codes[b, h].T)).amax(0)
                    best[:case["sink"]] = math.inf
                    ranked = sorted(range(blocks), key=lambda z, r=best.tolist(): (-r[z], z))
                    chosen = sorted(ranked[:top])
                    picked[b, h, i, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
                see = torch.zeros(case["n"], dtype=torch.bool, device="cuda")
                see[c["cut"]:] = True
                for z in chosen:
                    see[z * case["block"]:min((z + 1) * case["block"], c["cut"])] = True
                a = (x @ k[see].T) / math.sqrt(128.0)
                out[b, h * group:(h + 1) * group, i] = torch.softmax(a, 1) @ v[see]
    return [out, picked]
