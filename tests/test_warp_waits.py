"""Bounded waits end for a whole warp or for a thread alone, never for some lanes.

A bounded wait (mbar_wait, wait_or_abort) ends by each lane's own clock, so when the copy it
waits for lands as the limit runs out some lanes are told yes and others no. In code that a
whole warp runs, with warp-wide instructions behind it, that answer has to go through a vote
before anything depends on it. CPU: the kernels' sources are read: every wait whose answer
is used stands in a vote, goes into a variable that is voted on, or lies in a block that one
lane runs. GPU: waits that run out at any item of a decode call end it, with the status set.
"""
import os
import re

import pytest

from oracle import kvq_oracle as O

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quantized_sparse_kv_gb300", "csrc")
WAIT = re.compile(r"\b(?:mbar_wait|wait_or_abort)\s*\(")


def plain(text):
    """The source without comments, each character at its place."""
    blank = lambda m: re.sub(r"[^\n]", " ", m.group())  # noqa: E731
    return re.sub(r"//[^\n]*|/\*.*?\*/", blank, text, flags=re.S)


def unvoted_waits(text):
    """Lines of the waits whose answer decides for a lane alone."""
    text, out = plain(text), []
    for m in WAIT.finditer(text):
        start = max(text.rfind(c, 0, m.start()) for c in ";{}") + 1
        head = text[start:m.start()]
        if re.search(r"__device__", head) or not head.strip():
            continue  # a definition, or a wait whose answer nobody takes
        if re.search(r"^[^()]*\)\s*$|^\s*if\s*\([^()]*\)\s*$", head):
            continue  # the same, behind the head of a loop (cut at its semicolons) or an if
        if re.search(r"__(?:all|any)_sync\s*\(", head):
            continue
        # the headers of the blocks around it
        depth, i, one_lane = 0, m.start(), False
        while i > 0 and not one_lane:
            i -= 1
            if text[i] == "}":
                depth += 1
            elif text[i] == "{" and depth:
                depth -= 1
            elif text[i] == "{":
                j = max(text.rfind(c, 0, i) for c in ";{}") + 1
                one_lane = re.search(r"\bif\s*\(\s*lane == 0\s*\)\s*$", text[j:i]) is not None
        if one_lane:
            continue
        name = re.search(r"\b(\w+)\s*=(?!=)", head)
        if name and re.search(r"__(?:all|any)_sync\s*\([^;]*\b%s\b" % name.group(1),
                              text[m.start():m.start() + 600]):
            continue
        out.append(text.count("\n", 0, m.start()) + 1)
    return out


def test_the_reader_tells_them_apart():
    bad = "void f() { for (;;) { if (!mbar_wait(b, 0, l)) { break; } } }"
    assert unvoted_waits(bad) == [1]
    assert unvoted_waits("void f() {\n bool x = mbar_wait(b, 0, l);\n if (x) g();\n}") == [2]
    for good in ("void f() { mbar_wait(b, 0, l); }",
                 "void f() { for (int i = 0; i < 3; ++i) mbar_wait(b, 0, l); }",
                 "void f() { if (__any_sync(~0u, !mbar_wait(b, 0, l))) return; }",
                 "void f() { bool x = mbar_wait(b, 0, l); if (__any_sync(~0u, !x)) return; }",
                 "void f() { if (lane == 0) { for (;;) { if (!mbar_wait(b, 0, l)) break; } } }",
                 "// if (!mbar_wait(b, 0, l))\n"):
        assert unvoted_waits(good) == [], good


# (the candidate union's loaders wait for slots of a thread's own, with nothing warp-wide behind)
OWN = {"attend_candidates.cu": 1}


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_a_warp_leaves_a_wait_as_one(name):
    with open(os.path.join(CSRC, name)) as f:
        assert len(unvoted_waits(f.read())) == OWN.get(name, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,length", [(1, 2048), (9, 700)])
def test_decode_waits_that_run_out_at_any_item_end_the_call(batch, length):
    torch = pytest.importorskip("torch")
    from quantized_sparse_kv_gb300 import kvq
    gen = torch.Generator(device="cuda").manual_seed(batch)
    k = torch.randn((batch, 2, length, 128), generator=gen, device="cuda").bfloat16()
    v = torch.randn((batch, 2, length, 128), generator=gen, device="cuda").bfloat16()
    q = torch.randn((batch, 16, 1, 128), generator=gen, device="cuda").bfloat16()
    call = kvq.Attend(kvq.pack(k, v, 128, "bf16"), q, out_dtype="f32")
    want = call.run().clone()
    for item in range(24):
        kvq.debug_set(2_000_000, item)  # 2 ms; this item is never copied
        try:
            call.run()
            assert kvq.read_status(call.status) & kvq.DEV_TIMEOUT
        finally:
            kvq.debug_set(0, -1)
        call.status.zero_()
    got = call.run()
    assert kvq.read_status(call.status) == 0 and torch.equal(got, want)
    ref, _ = O.attend(q.float().cpu().numpy(),
                      O.pack(k.float().cpu().numpy(), v.float().cpu().numpy(), 128, "bf16"))
    # (the tensor-core decode path against the oracle: five factors rounded to 11 bits)
    assert O.rel_l2(got.cpu().numpy(), ref) <= 5e-3
