"""The checked build's region check (bit 2) in the copies of sequences and in
the chunk kernel: an address outside the cache region is reported in that
cache's word and not accessed, all others are as ever."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def result():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_region_run.py")], capture_output=True, text=True,
                       env=dict(os.environ, KIVI_DEBUG_CHECKS="1"), timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = json.loads([line for line in r.stdout.splitlines() if line.startswith("{")][-1])
    assert res["lib"] == "libkivi_debug.so"
    return res


@pytest.mark.parametrize("what", ["fork", "cycle", "onto"])
def test_reorder(result, what):
    assert result[f"{what}_flag"] == 4 and result[f"{what}_same"] and result[f"{what}_after"] == 0, result


@pytest.mark.parametrize("what", ["from", "into"])
def test_copy(result, what):
    assert result[f"{what}_flag"] == 4 and result[f"{what}_same"] and result[f"{what}_clean"] == 0, result


@pytest.mark.parametrize("what", ["sinks", "ring", "frozen"])
def test_chunks(result, what):
    assert result[f"chunk_{what}_flag"] == 4 and result[f"chunk_{what}_after"] == 0, result
