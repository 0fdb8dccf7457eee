"""Host helpers of bench.py that need no GPU: the DRAM traffic recorded for a
kernel holds while that kernel's own sources do, whatever is added beside them."""
import json
import os
import shutil

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FOLDER = os.path.join("turboquant_kv_cache_tq_gb300", "csrc")


@pytest.fixture
def csrc(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(ROOT, FOLDER), tmp_path / FOLDER)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path / FOLDER


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_UNITS))
def test_other_kernels_do_not_change_a_kernels_hash(csrc, kernel):
    before = bench.kernel_source_hash(kernel)
    (csrc / "tq_another.cu").write_text('#include "tq_kernels.cuh"\nint another;\n')
    for name in ("tq_tree_attention.cuh", "tq_evict.cu", "tq_lloyd.cu"):
        (csrc / name).write_text((csrc / name).read_text() + "\nint more;\n")
    assert bench.kernel_source_hash(kernel) == before


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_UNITS))
@pytest.mark.parametrize("name", ["tq_kernels.cuh", "tq_decode_bulk.cuh", "tq_tables.cuh", "tq_abi.cu"])
def test_what_a_kernel_includes_changes_its_hash(csrc, kernel, name):
    before = bench.kernel_source_hash(kernel)
    (csrc / name).write_text((csrc / name).read_text() + "\nint more;\n")
    assert bench.kernel_source_hash(kernel) != before


def test_recorded_traffic_is_found_by_its_kernel(csrc, tmp_path, monkeypatch):
    path = tmp_path / "traffic.json"
    monkeypatch.setattr(bench, "PROFILE_TRAFFIC", str(path))
    path.write_text(json.dumps({"encode_kernel@w": {"source_hash": bench.kernel_source_hash("encode_kernel"),
                                                    "dram_bytes_per_launch": 7}}))
    assert bench.profiled_traffic("encode_kernel@w") == 7
    assert bench.profiled_traffic("decode_bulk_kernel@w") is None
    (csrc / "tq_attention.cuh").write_text((csrc / "tq_attention.cuh").read_text() + "\nint more;\n")
    assert bench.profiled_traffic("encode_kernel@w") == 7
    (csrc / "tq_encode_d64.cu").write_text((csrc / "tq_encode_d64.cu").read_text() + "\nint more;\n")
    assert bench.profiled_traffic("encode_kernel@w") is None


def test_recorded_kernels_are_known():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        for key in json.load(f):
            assert key.startswith("_") or key.split("@")[0] in bench.KERNEL_UNITS, key
