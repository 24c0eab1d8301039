"""The bench's DRAM traffic figure is that of an ncu capture, for as long as
the sources of the captured kernels stay as they were: the figure that is
kept belongs to the present sources, other kernels' sources do not matter, and
those that the captured kernels are built from do (no GPU needed)."""
import os
import shutil
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402

CSRC = os.path.join(bench.ROOT, "kv_cache_quantization_hqmq_b200", "csrc")


def test_the_kept_figure_is_of_the_present_sources():
    n, note = bench.captured_traffic()
    assert n is not None, note
    # 1 x 8 x 131072 x 128 bf16 read at least once, codes and list written: 388 MB; never read three times
    assert 300e6 < n < 900e6


@pytest.mark.parametrize("name,matters", [
    ("encode_spec.cu", True), ("med3_window.cu", True), ("search.cu", True), ("decode.cu", True), ("search.cuh", True),
    ("med3_window.cuh", True), ("hqmq_device.cuh", True), ("paged_attention.cu", False), ("paged.cuh", False),
    ("norm_rope.cu", False), ("joint.cu", False)])
def test_which_sources_the_figure_depends_on(tmp_path, name, matters):
    before = bench.kernel_sources_sha256()
    copy = tmp_path / "csrc"
    shutil.copytree(CSRC, copy)
    assert bench.kernel_sources_sha256(str(copy)) == before
    with open(copy / name, "a") as f:
        f.write("// changed\n")
    assert (bench.kernel_sources_sha256(str(copy)) != before) == matters
