"""Run the calls around a decoding step once through one build of the library.

python tests/debug_operator_cases.py LIB OUT.npz

Loads LIB (libkvq.so or libkvq_debug.so), runs small seeded cases of rotary
positions, tree attention (tensor-core and fp32 kernels), block summaries and
their values, the choice of blocks and attention over them, and saves every
output (as raw bytes) and every status word. test_operators_debug compares
the files of the two builds.
"""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def main(lib_path: str, out_path: str) -> None:
    import torch

    from quantized_sparse_kv_gb300 import kvq

    lib = kvq.load_library(lib_path)
    res = {"checks": np.array(lib.kvq_debug_checks())}
    gen = torch.Generator(device="cuda").manual_seed(11)

    def rand(*shape, dt=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    def keep(name, t, status=None):
        t = t.detach().contiguous()
        if t.dtype == torch.bfloat16:
            t = t.view(torch.int16)
        res[name] = t.cpu().numpy()
        if status is not None:
            res["status_" + name] = np.array(kvq.read_status(status))

    # rotary positions: both layouts, partial, scalar pairs, strided rows, fp32
    for i, (layout, r, d, dt) in enumerate((("half", 128, 128, torch.bfloat16),
                                            ("half", 30, 64, torch.bfloat16),
                                            ("interleaved", 48, 96, torch.float32),
                                            ("half", 64, 256, torch.float32))):
        rows = rand(2, 19, 7, d, dt=dt)
        call = kvq.Rope(kvq.RopePlan(r, layout=layout), rows[:, :, :4].transpose(1, 2),
                        rows[:, :, 4:6].transpose(1, 2),
                        torch.arange(38, device="cuda").view(2, 19) * 1001,
                        v=rows[:, :, 6:].transpose(1, 2))
        status = kvq.new_status()
        kvq._check(lib.kv_rope(*call._args[:-1], kvq._ptr(status), kvq._stream()), "kv_rope")
        for j, o in enumerate(call.out):
            keep(f"rope{i}_{j}", o, status)

    def cache(b, h, n, d, recent, kwin="bf16", vwin="bf16", reserve=None):
        dt = torch.float32 if kwin == "f32" else torch.bfloat16
        return kvq.pack(rand(b, h, n, d, dt=dt), rand(b, h, n, d, dt=dt), recent, kwin, vwin,
                        reserve=reserve)

    par = torch.tensor([[-1, 0, 0, 1, 3, -1, 5], [-1, -1, 1, 2, -2, -2, -2]], dtype=torch.int32,
                       device="cuda")
    for i, (n, recent, d, kwin, hq, reserve) in enumerate((
            (700, 75, 128, "bf16", 16, None), (257, 0, 128, "bf16", 10, (12, 40)),
            (4000, 128, 128, "bf16", 80, None), (150, 40, 64, "f32", 4, None),
            (90, 90, 128, "mxfp8", 8, None))):
        c = cache(2, 2, n, d, recent, kwin, "f32" if kwin == "f32" else "bf16", reserve)
        dt = torch.float32 if kwin == "f32" else torch.bfloat16
        k, v = rand(2, 2, 7, d, dt=dt), rand(2, 2, 7, d, dt=dt)
        v[:, :, 2, 1] = torch.inf
        call = kvq.AttendTree(c, rand(2, hq, 7, d, dt=dt), k, v, par, out_dtype="f32")
        keep(f"tree{i}", call.run(), call.status)

    for i, (n, recent, d, block, top, hq, nq, dt) in enumerate((
            (3000, 128, 128, 64, 9, 16, 1, torch.bfloat16), (1000, 77, 128, 32, 40, 14, 3, torch.bfloat16),
            (700, 0, 64, 128, 2, 4, 2, torch.float32), (100000, 1, 128, 32, 33, 16, 1, torch.bfloat16))):
        c = cache(2, 2, n, d, recent, reserve=(-(-(n - recent) // 32) + 3, recent + 2))
        s = kvq.BlockSummary(c, block).update()
        keep(f"values{i}", s.values(1))
        status = kvq.new_status()
        kvq._check(lib.kv_block_summary(c.ref, s.ref, 0, kvq._ptr(status), kvq._stream()),
                   "kv_block_summary")
        keep(f"codes{i}", s.codes[:, :, :s.blocks], status)
        call = kvq.AttendBlocks(c, rand(2, hq, nq, d, dt=dt), s, top, n_sink=1, out_dtype="f32")
        keep(f"blocks{i}", call.run(), call.status)
        keep(f"selected{i}", call.selected)

    torch.cuda.synchronize()
    np.savez(out_path, **res)


if __name__ == "__main__":
    main(sys.argv[1], sys.argv[2])
