"""The row operators' index checks (debug-bounds build) stay silent on their GPU test cases (GPU): list, group, bin,
slice and token indices of filtered sampling, top logits and distillation.  The tests run against
libspecverify_debug.so in a child process, which at its end asks the library for what the checks recorded."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import sys, pytest, torch
rc = pytest.main(sys.argv[1:])
import speculative_decoding_verification_40_gb300 as S
assert S.LIB_PATH.endswith("libspecverify_debug.so"), S.LIB_PATH
torch.cuda.synchronize()
status = S.check_status(raise_on_error=False)
print("status of the index checks:", status)
sys.exit(rc or status)
"""


@pytest.mark.parametrize("files,pick", [
    (["tests/test_gpu_filtered.py", "tests/test_gpu_filtered_borders.py", "tests/test_gpu_top_logits.py"],
     "sizes or list or order or ties or borders and not levels"),
    (["tests/test_gpu_distill.py", "tests/test_gpu_distill_ranges.py", "tests/test_gpu_train_and_serve.py"],
     "sizes or far or masked or invalid or place or hold or record"),
])
def test_row_operators_under_index_checks(files, pick):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location(
        "specverify_build", os.path.join(ROOT, "speculative_decoding_verification_40_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build(debug_bounds=True)
    env = dict(os.environ, SPECVERIFY_DEBUG_BOUNDS="1", PYTHONPATH=ROOT)
    cmd = [sys.executable, "-c", CHILD, "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files, "-k", pick]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert "passed" in tail and "status of the index checks: 0" in tail, tail
