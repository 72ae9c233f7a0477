"""The binding serves the host planner, the versions and the sizes without
torch: a process that cannot import it loads the library all the same."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None  # `import torch` raises ImportError
import numpy as np
import mqa_decode_attention_paged_gb300 as pkg
from mqa_decode_attention_paged_gb300 import _binding as mqa
assert pkg.abi_version() == mqa.lib.mqa_abi_version()
assert pkg.status_string(0)
assert pkg.num_kv_splits(5000, 152) >= 1
assert pkg.gqa_window_decode_workspace_bytes(3, 1, 32, 8, 128, 5) == 3 * 5 * 8 * 4 * 129 * 4 + 3 * 8
bt = np.arange(8, dtype=np.int32).reshape(2, 4)
table, lens = mqa.dcp_shard(bt, np.array([40, 17], dtype=np.int32), 16, 2, 0, "round_robin")
assert lens.tolist() == [24, 16], lens
try:
    pkg.gqa_window_decode
except ImportError:
    pass  # the call takes torch tensors
else:
    raise AssertionError
try:
    mqa.no_such_name
except AttributeError:
    print("ok")
"""


def test_binding_without_torch():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
