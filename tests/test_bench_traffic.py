"""The kernel source that a committed traffic figure is valid for: every file that the chunk kernels are made of."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join("rl_fine_tuning_gb300", "csrc")


@pytest.mark.parametrize("name", ["tc_kernels.cu", "tc_pair.cuh", "ptx.cuh", "internal.h", "small_kernels.cu"])
def test_a_change_to_the_chunk_kernels_source_changes_its_hash(name, tmp_path, monkeypatch):
    """The pair engine and its dH and dW traits live in headers: a change there makes an older capture invalid."""
    shutil.copytree(os.path.join(ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_source_hash()
    assert before == bench.kernel_source_hash()
    with open(tmp_path / CSRC / name, "a") as f:
        f.write("// changed\n")
    assert bench.kernel_source_hash() != before


def test_the_hash_leaves_other_kernels_out(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_source_hash()
    for name in ("head_tc.cu", "head_kernels.cu", "head_abi.cu", "head.h"):
        with open(tmp_path / CSRC / name, "a") as f:
            f.write("// changed\n")
    assert bench.kernel_source_hash() == before
