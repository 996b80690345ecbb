"""Where the CTA-pair GEMM puts a split tile's partial tiles and output boxes
in its idle ring, for every width, stage form, epilogue and number of parts:
nothing may reach past the ring into the barriers and operands behind it.
The arithmetic is the kernels' own header, compiled here.  CPU only."""
import ctypes
import os
import subprocess

import pytest

from fp16_tensor_core_gb300 import build as dg_build

WIDTHS = (128, 160, 192, 224, 256)


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    where = tmp_path_factory.mktemp("smem")
    source = where / "probe.cpp"
    source.write_text("""#include "gemm_smem.h"
extern "C" {
int limit() { return dg::kSmemLimit; }
int max_parts() { return dg::kPairMaxParts; }
int stages(int bn, int kps, int fused) { return dg::pair_stages_for(bn, kps, fused != 0); }
int ring(int bn, int kps, int fused) { return dg::pair_ring_bytes(bn, kps, fused != 0); }
int behind(int bn, int fused) { return dg::pair_staging_bytes(fused != 0) + (fused ? dg::columns_bytes(bn) : 0); }
int in_ring(int ring, int bn, int parts) { return dg::pair_parts_in_ring(ring, bn, parts); }
int boxes_at(int bn, int parts) { return dg::pair_boxes_at(bn, parts); }
}
""")
    lib = where / "probe.so"
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", dg_build.CSRC, str(source), "-o", str(lib)], check=True)
    return ctypes.CDLL(os.fspath(lib))


@pytest.mark.parametrize("bn", WIDTHS)
@pytest.mark.parametrize("kps", [1, 2])
@pytest.mark.parametrize("fused", [0, 1])
def test_what_a_tile_is_finished_with_fits(sizes, bn, kps, fused):
    ring = sizes.ring(bn, kps, fused)
    assert sizes.stages(bn, kps, fused) >= 2
    # the alignment's slack, the ring, the barriers, staging boxes and columns
    assert 1024 + ring + 1024 + sizes.behind(bn, fused) <= sizes.limit()
    partial, boxes = 128 * bn * 4, 128 * bn * 2     # FP32 partial tile; 16-bit output, as 32 x 32 boxes
    assert sizes.boxes_at(bn, 1) == 0 and boxes <= ring     # whole tiles, and partial tiles read from L2
    assert sizes.max_parts() == 4
    for parts in range(2, sizes.max_parts() + 1):
        at = sizes.boxes_at(bn, parts)
        assert at % 1024 == 0 and at >= (parts - 1) * partial, (parts, "boxes over partial tiles that are still read")
        assert not sizes.in_ring(ring, bn, parts) or at + boxes <= ring, (parts, at, boxes, ring)
    assert sizes.in_ring(ring, bn, 2)               # two parts always take the ring


def test_the_parts_that_do_not_fit(sizes):
    """Three partial tiles of 128 columns fill 192 KB by themselves; two of 160
    and of 192 leave too little for the boxes with one K block a stage."""
    for bn, kps, fused, parts in ((128, 1, 0, 4), (128, 2, 1, 4), (160, 1, 1, 3), (192, 1, 0, 3), (256, 2, 1, 3)):
        assert not sizes.in_ring(sizes.ring(bn, kps, fused), bn, parts), (bn, kps, fused, parts)
