"""The DRAM figures of the benchmark belong to the sources as they are, and stay with them while
only operators around the FFN, comments or the names of timing events change."""
import json
import os
import shutil

import pytest

import bench
from activation_sparse_transformer_gate_gb300 import _build


@pytest.fixture
def copy(tmp_path):
    d = tmp_path / "csrc"
    shutil.copytree(_build.CSRC, d)
    return d


def change(path, old, new):
    text = path.read_text(encoding="utf-8")
    assert old in text
    path.write_text(text.replace(old, new, 1), encoding="utf-8")


def test_the_figures_are_of_these_sources():
    d = json.load(open(os.path.join(bench.ROOT, "profiles", "traffic.json")))
    assert d and {e["source_hash"] for e in d.values()} == {bench.kernel_source_hash()}
    kernel, workload, mode = next(iter(d)).split("|")
    assert bench.traffic_for(kernel, workload, mode == "train") > 0


def test_other_operators_do_not_count(copy):
    before = bench.kernel_source_hash()
    assert bench.kernel_source_hash(str(copy)) == before
    for f in set(_build.SOURCES) - set(_build.FFN_SOURCES):
        (copy / f).write_text("int another;\n")
    (copy / "another.cuh").write_text("int another;\n")
    change(copy / "kernels.h", "  KID_COUNT = ", "  KID_ANOTHER = 1000,\n  KID_COUNT = ")
    change(copy / "twell_abi.cu", '"adamw_step"', '"adamw_step", "another"')
    change(copy / "common.cuh", "// ---- element conversions", "// another comment\n// ---- element conversions")
    assert bench.kernel_source_hash(str(copy)) == before


@pytest.mark.parametrize("f", ["updown.cu", "tc_gemm.cu", "common.cuh", "gather.cuh", "tcgen05.cuh",
                               "kernels.h"])
def test_the_ffn_counts(copy, f):
    with open(copy / f, "a", encoding="utf-8") as out:
        out.write("int another;\n")
    assert bench.kernel_source_hash(str(copy)) != bench.kernel_source_hash()
