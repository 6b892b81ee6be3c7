"""The operators for drafted tokens on the bounds-checked build (kv_cache_compression_gb300.build.build(checked=True)), with a status
word in every call: tiles, parts and appended rows, whose places follow from lengths and schedules, are checked before the access,
and a violation skips it and is reported. A child process loads that build and runs the operators' parity tests on it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

SUBSET = ["tests/test_gpu_tree.py", "tests/test_gpu_rows.py", "tests/test_gpu_tree_edges.py", "tests/test_gpu_draft_extremes.py"]


def test_the_operators_for_drafted_tokens_on_the_bounds_checked_build(gpu_device):
    from kv_cache_compression_gb300 import build as kbuild
    assert os.path.exists(kbuild.build(checked=True))
    env = dict(os.environ, SNAPKV_CHECKED="1")
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                          "-p", "tests.watch_draft_status", *SUBSET],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert run.returncode == 0, run.stdout[-4000:] + run.stderr[-2000:]
    assert " passed" in run.stdout
