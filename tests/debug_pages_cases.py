"""Run the paged cache's calls once through one build of the library.

python tests/debug_pages_cases.py LIB OUT.npz

Loads LIB (libkvq.so or libkvq_debug.so), takes small seeded requests through tables,
appends, values read back and attention (both kernels), and saves every output (as raw
bytes) and every status word. test_pages_edges compares the files of the two builds.
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
    gen = torch.Generator(device="cuda").manual_seed(21)

    def keep(name, t, status=None):
        t = t.detach().contiguous()
        if t.dtype == torch.bfloat16:
            t = t.view(torch.int16)
        res[name] = t.cpu().numpy()
        if status is not None:
            res["status_" + name] = np.array(kvq.read_status(status))

    steps = [[300, 40, 0, 129], [1, 1, 700, 0], [1, -1, 1, 64], [1, 97, 1, 1]]
    for i, (page, window, hk, hq, d, dt, wdt) in enumerate((
            (64, 128, 2, 16, 128, torch.bfloat16, "bf16"),
            (32, 33, 1, 5, 64, torch.float32, "bf16"),
            (128, 0, 3, 3, 96, torch.float32, "f32"),
            (32, 64, 2, 18, 128, torch.bfloat16, "f32"),
            (64, 100, 1, 12, 256, torch.bfloat16, "bf16"))):
        state = kvq.PageState(4, 60, page, 30, window)
        cache = kvq.PagedCache(state, hk, d, wdt)
        cache.pool.zero_()
        cache.ring.zero_()
        for j, new in enumerate(steps):
            rows = sum(max(0, n) for n in new) + j
            plan = kvq.page_tables(state, torch.tensor(new, device="cuda"), rows)
            x = torch.randn((rows, 2 * hk, d), generator=gen, device="cuda").to(dt)
            put = kvq.AppendPages(cache, plan, x[:, :hk], x[:, hk:])
            put.run()
            tag = f"{i}_{j}"
            keep("slots" + tag, plan.row_slot, plan.status)
            keep("positions" + tag, plan.positions)
            keep("work" + tag, plan.work[:int(plan.counts[1]), :6])
            keep("lengths" + tag, state.lengths)
            keep("pool" + tag, cache.pool, put.status)
            keep("ring" + tag, cache.ring)
            vals = kvq.PageValues(cache, plan.row_slot, plan.positions)
            vals.run()
            keep("keys" + tag, vals.k, vals.status)
            keep("values" + tag, vals.v)
            q = torch.randn((rows, hq, d), generator=gen, device="cuda").to(dt)
            call = kvq.AttendPages(cache, q, plan.row_slot, plan.positions, out_dtype="f32")
            keep("rows" + tag, call.run(), call.status)
            call = kvq.AttendPages(cache, q[:4])
            keep("all" + tag, call.run(), call.status)
    np.savez(out_path, **res)


if __name__ == "__main__":
    main(sys.argv[1], sys.argv[2])
