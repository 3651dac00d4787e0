"""Host-side check of the shared-memory plans of the few-token products (no GPU needed).

Compiles tests/host/moe_plan_check.cu -- which includes the kernels' source and calls their planners -- with nvcc for the
host, and runs it over about a million plans."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_every_product_plan_is_in_range(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = tmp_path / "moe_plan_check"
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "tp_reduce_moe_gb300", "csrc"),
                    os.path.join(HERE, "host", "moe_plan_check.cu"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:]
    assert " 0 bad" in r.stdout


def test_ranges_cover_every_tile_once():
    """How a job's segments are cut into sixteen ranges, and which parts a tile's sum takes: the kernels' arithmetic."""
    for count in list(range(1, 33)):
        for length in (1, 2, 3, 5, 14, 16, 55, 56, 64, 127, 128):
            total = count * length
            ranges = [(total * w // 16, total * (w + 1) // 16) for w in range(16)]
            parts = {}
            for w, (f0, f1) in enumerate(ranges):
                for f in range(f0, f1):
                    parts[w, f // length] = parts.get((w, f // length), 0) + 1
            places = [w + tile for w, tile in parts]
            assert len(set(places)) == len(places) and max(places) < count + 16
            for tile in range(count):
                lo, hi = tile * length, (tile + 1) * length
                first = tile * 16 // count
                taken = [w for w in range(first, 16)
                         if total * w // 16 < hi and total * (w + 1) // 16 > lo and total * (w + 1) // 16 > total * w // 16]
                assert sum(parts[w, tile] for w in taken) == length
