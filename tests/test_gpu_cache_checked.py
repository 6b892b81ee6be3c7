"""The cache operators on the bounds-checked build (kv_cache_compression_gb300.build.build(checked=True)): the
tiles that attention copies, the cache rows that quantisation writes and the slots that an eviction moves, which
follow from lengths, schedules and lists, are checked before the access, and a violation skips it and is reported.
A child process loads that build and runs the operators' parity tests on it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

SUBSET = ["tests/test_gpu_cache_q4.py", "tests/test_gpu_cache_evict.py",
          "tests/test_gpu_cache_attend.py::test_schedules_with_empty_and_uneven_sequences",
          "tests/test_gpu_cache_attend.py::test_random_shapes", "tests/test_gpu_cache_attend.py::test_long_and_wide",
          "tests/test_gpu_cache_attend.py::test_lengths_outside_the_cache"]


def test_the_cache_operators_on_the_bounds_checked_build(gpu_device):
    from kv_cache_compression_gb300 import build as kbuild
    assert os.path.exists(kbuild.build(checked=True))
    env = dict(os.environ, SNAPKV_CHECKED="1")
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *SUBSET],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert run.returncode == 0, run.stdout[-4000:] + run.stderr[-2000:]
    assert " passed" in run.stdout


# The joining launch: parts of cut heads, logits and scores, turns over long caches, the table of sums of large batches.
JOINS = ["tests/test_gpu_cache_extremes.py", "tests/test_gpu_cache_nonfinite.py",
         "tests/test_gpu_cache_attend.py::test_joins_of_every_size",
         "tests/test_gpu_cache_attend.py::test_dense_ragged_lengths", "tests/test_gpu_cache_attend.py::test_q4_ragged_lengths"]


def test_joins_and_the_largest_shapes_on_the_bounds_checked_build(gpu_device):
    """With a status word in every call (tests/watch_status.py), as the tests themselves pass none."""
    from kv_cache_compression_gb300 import build as kbuild
    assert os.path.exists(kbuild.build(checked=True))
    env = dict(os.environ, SNAPKV_CHECKED="1")
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                          "-p", "tests.watch_status", *JOINS, *SUBSET],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert run.returncode == 0, run.stdout[-4000:] + run.stderr[-2000:]
    assert " passed" in run.stdout
