"""The launch shape of the norm's gradient over all widths, compiled from its
own header: the ring serves every row that its kernels' registers hold."""
from __future__ import annotations

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixed_precision_dense_02_gb300", "csrc")
MAIN = """
#include <stdio.h>
#include "norm_shape.h"
int main() {
  for (int t = 2; t <= 3; ++t)
    for (long v = 1; v <= 2100; ++v) {
      const mmagb::NormBackShape s = mmagb::norm_back_shape(v, t);
      printf("%d %ld %d %d %d %d\\n", t, v, s.vpt, s.threads, s.per_sm, s.stages);
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
    for t, v, vpt, threads, per_sm, stages in shapes:
        assert (stages >= 2) == (v <= 2048), (t, v)


def test_blocks_fit_an_sm(shapes):
    for t, v, vpt, threads, per_sm, stages in shapes:
        if v > 2048:
            continue
        assert vpt in (1, 2, 4) and threads % 32 == 0 and threads <= 512
        assert threads * vpt >= v and 2 <= stages <= 4
        assert per_sm * threads * (128 if vpt == 4 else 64) <= 65536
        # a KB per block and the barriers and sums beside the ring
        assert per_sm * (stages * v * 16 * t + 1024 + 1024) <= 228 * 1024
        assert stages * v * 16 * t <= 220 * 1024
        assert per_sm <= 3
