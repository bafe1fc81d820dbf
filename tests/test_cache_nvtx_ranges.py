"""The paged-cache entry points open NVTX ranges named after themselves, as the scoring and
selection ones do (checked on the CPU, on calls that the host rejects)."""

import os
import shutil
import subprocess
import sys

import pytest

from test_nvtx_ranges import CUDA_INC, INJECTION_C, ROOT

CALLS = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
import kv_cache_eviction_scores_b200 as dk
L = dk.lib()
res = [L.dropkv_cache_write(None, None, None, None), L.dropkv_cache_read(None, None, None, None),
       L.dropkv_cache_attention(None, None, None, 0, None, None)]
assert all(r == dk.ERR_ARG for r in res), res
print("ok")
"""


def test_cache_entry_points_open_named_nvtx_ranges(tmp_path):
    if shutil.which("gcc") is None or not os.path.exists(
            os.path.join(CUDA_INC, "nvtx3", "nvToolsExt.h")):
        pytest.skip("needs gcc and the NVTX3 headers")
    src, so, log = tmp_path / "inject.c", tmp_path / "libinject.so", tmp_path / "ranges.log"
    src.write_text(INJECTION_C)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-I", CUDA_INC, str(src), "-o", str(so)],
                   check=True)
    env = dict(os.environ, NVTX_INJECTION64_PATH=str(so), DROPKV_NVTX_LOG=str(log))
    out = subprocess.run([sys.executable, "-c", CALLS, ROOT], env=env, capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0 and "ok" in out.stdout, out.stderr[-2000:]
    names = ["dropkv_cache_write", "dropkv_cache_read", "dropkv_cache_attention"]
    assert log.read_text().splitlines() == [x for n in names for x in (f"push {n}", "pop")]
