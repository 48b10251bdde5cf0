"""The bounds-checked build (libkvq_debug.so) on the calls around a decoding
step: the same bytes as the release build and nothing flagged on valid inputs
(tests/debug_operator_cases.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_both_builds_agree(tmp_path):
    from quantized_sparse_kv_gb300 import kvq
    files = []
    for lib in (kvq.LIB_PATH, kvq.DEBUG_LIB_PATH):
        out = str(tmp_path / (os.path.basename(lib) + ".npz"))
        r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_operator_cases.py"),
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
