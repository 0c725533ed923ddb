"""Threads of the 8-bit quantiser, compiled as host code."""

from __future__ import annotations

import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = r"""
#include <cstdio>
#include "int8_plan.h"
int main() {
  int rows, K, f32, sms;
  while (std::scanf("%d %d %d %d", &rows, &K, &f32, &sms) == 4) std::printf("%d\n", sesg::quantize_threads(rows, K, f32, sms));
}
"""


def test_few_rows_are_few_for_the_device(tmp_path):
    """Up to two rows a SM, whatever the device's number of SMs, a row is spread over as many threads as have two loads."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "q.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-I", f"{ROOT}/sparse_expert_swiglu_gb300/csrc", str(tmp_path / "q.cpp"), "-o",
                    str(tmp_path / "q")], check=True)
    want = {}
    for sms in (152, 148, 36):
        for f32 in (0, 1):
            keep = 4 if f32 else 8
            for K in (16, 512, 1008, 4096, 14336, 65536):
                few = next(t for t in (32, 64, 128, 256, 512, 1024) if t == 1024 or t * 2 >= K // 8)
                many = next(t for t in (32, 64, 128, 256, 512, 1024) if t == 1024 or t * keep >= K // 8)
                for rows in (1, 2 * sms):
                    want[rows, K, f32, sms] = few
                for rows in (2 * sms + 1, 100000):
                    want[rows, K, f32, sms] = many
    text = "".join("%d %d %d %d\n" % s for s in want)
    out = subprocess.run([str(tmp_path / "q")], input=text, capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == list(want.values())
