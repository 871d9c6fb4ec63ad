"""Rules of the grouped and FP8 matmul sources that no result shows: the compiler
usually brings a warp's lanes back together, the language does not promise it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_moe_layer_limited_b200", "csrc")
FILES = ["grouped_matmul.cu", "grouped_matmul_fp32.cu", "matmul_narrow.cu", "matmul_dw_small.cu",
         "matmul_fp8.cu"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_aligned_barriers_meet_whole_warps(name):
    """Cluster barriers go through the form that gathers the warp's lanes first, and so does the
    epilogue's named barrier."""
    text = source(name)
    assert not re.search(r"\bcluster_sync_all\(|barrier\.cluster", text)
    for m in re.finditer(r'"bar\.sync', text):
        assert re.search(r"__syncwarp\(\);\s*asm volatile\($", text[:m.start()])


def test_the_gathering_form_does():
    text = source("matmul_util.cuh")
    assert re.search(r"mm_cluster_sync\(\) \{\s*__syncwarp\(\);\s*cluster_sync_all\(\);\s*\}", text)
