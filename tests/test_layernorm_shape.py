"""The launch shapes of the layer norm and its gradient over all widths, compiled from
their own header: a ring of two rows and more, within what an SM has."""
from __future__ import annotations

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixed_precision_dense_02_gb300", "csrc")
MAIN = """
#include <stdio.h>
#include "norm_shape.h"
void put(int back, int t, long v, mmagb::NormRingShape s) {
  printf("%d %d %ld %d %d %d %d\\n", back, t, v, s.vpt, s.threads, s.per_sm, s.stages);
}
int main() {
  for (long v = 1; v <= 2100; ++v) {
    for (int t = 1; t <= 2; ++t) put(0, t, v, mmagb::layernorm_shape(v, t));
    for (int t = 2; t <= 3; ++t) put(1, t, v, mmagb::layernorm_back_shape(v, t));
  }
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    d = tmp_path_factory.mktemp("shape")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / "main")],
                   check=True)
    out = subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_every_width_has_a_ring(shapes):
    for back, t, v, vpt, threads, per_sm, stages in shapes:
        assert (vpt > 0) == (v <= 2048), (back, t, v)


def test_blocks_fit_an_sm(shapes):
    # the kernels' launch bounds and registers a thread (csrc/layernorm.cu)
    most = {(0, 1): (512, 128), (0, 2): (512, 128), (0, 4): (512, 128),
            (1, 1): (128, 64), (1, 2): (384, 80), (1, 4): (512, 128)}
    for back, t, v, vpt, threads, per_sm, stages in shapes:
        if v > 2048:
            continue
        threads_most, registers = most[back, vpt]
        assert threads % 32 == 0 and threads <= threads_most and threads * vpt >= v
        assert 2 <= stages <= 4 and per_sm >= 1
        assert per_sm * threads * registers <= 65536, (back, t, v)
        assert stages * v * 16 * t <= 220 * 1024
        # a KB per block and the barriers and sums beside the ring
        assert per_sm * (stages * v * 16 * t + 1024 + 1024) <= 228 * 1024, (back, t, v)
