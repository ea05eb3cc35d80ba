"""The profiled counters that bench.py reports beside the GEMMs' rate: they
belong to the GEMM code of this tree, and the rest of the library may change
without dropping them."""

import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

BUILD = "quantize_grouped_gemm_amd/build.py"


def test_recorded_counters_are_this_trees():
    """After a change to the GEMM's code: take the counters again (the commands
    stand in the files) and record bench.gemm_source_hash() with them."""
    assert bench._measured_traffic() is not None, bench.TRAFFIC_FILE
    assert bench._measured_mfma() is not None, bench.MFMA_FILE


@pytest.mark.parametrize("old,new,same", [
    ('SOURCES = ["mx_quant.hip"', 'SOURCES = ["another.hip", "mx_quant.hip"', True),
    ('"""Builds libmxfp8.so', '"""Compiles libmxfp8.so', True),
    ('"-O3"', '"-O2"', False),
    ('ARCH = "gfx950"', 'ARCH = "gfx942"', False)])
def test_only_the_flags_of_the_build_file_count(tmp_path, monkeypatch, old, new, same):
    for rel in bench.GEMM_SOURCES:
        dst = tmp_path / rel
        dst.parent.mkdir(parents=True, exist_ok=True)
        shutil.copy(os.path.join(ROOT, rel), dst)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    base = bench.gemm_source_hash()
    text = (tmp_path / BUILD).read_text()
    assert old in text
    (tmp_path / BUILD).write_text(text.replace(old, new, 1))
    assert (bench.gemm_source_hash() == base) == same
