"""pkv_bm_evict_batch is all or nothing also where host memory runs out (CPU only)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_eviction_survives_every_failed_allocation(tmp_path):
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if not os.path.isdir(cuda):
        pytest.skip("no CUDA headers")
    exe = str(tmp_path / "block_manager_alloc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wno-mismatched-new-delete", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "paged_kv_cache_373_b200", "csrc"), "-I", cuda,
                    os.path.join(HERE, "block_manager_alloc.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
