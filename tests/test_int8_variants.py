"""Every kernel of the 8-bit products on the tensor cores: sizes whose plans name each, and the registers that their warps
share out."""

from __future__ import annotations

import shutil
import subprocess

import pytest

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.conftest import ROOT  # noqa: E402
from tests.test_int8 import BF16, F16, F32, _linear_case, _linear_check  # noqa: E402
from tests.test_int8_plans import plan  # noqa: E402,F401

gpu = pytest.mark.gpu

# (CTAs of a product, whether clusters share a tile, gated, blocks of 16 columns of an epilogue warp): M, N, K
VARIANTS = {
    (1, 0, 0, 1): (18, 71, 32), (1, 0, 0, 2): (2476, 132, 144), (1, 0, 0, 4): (1644, 650, 144), (1, 0, 0, 6): (462, 12187, 272),
    (1, 0, 1, 1): (18, 71, 32), (1, 0, 1, 2): (34, 4867, 144), (1, 0, 1, 4): (194, 2797, 272), (1, 0, 1, 6): (129, 18043, 144),
    (1, 1, 0, 1): (18, 71, 1296), (1, 1, 0, 2): (226, 134, 6128), (1, 1, 0, 4): (592, 135, 5792), (1, 1, 0, 6): (1895, 258, 6608),
    (1, 1, 1, 1): (18, 71, 1296), (1, 1, 1, 2): (37, 457, 4704), (1, 1, 1, 4): (67, 826, 5744), (1, 1, 1, 6): (137, 947, 16304),
    (2, 0, 0, 4): (396, 2765, 528), (2, 0, 0, 6): (134, 12954, 704), (2, 0, 1, 4): (140, 3452, 688), (2, 0, 1, 6): (131, 6661, 1024),
    (2, 1, 0, 4): (1226, 131, 3568), (2, 1, 0, 6): (137, 3367, 11184), (2, 1, 1, 4): (393, 341, 3424), (2, 1, 1, 6): (149, 1608, 11984)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def test_sizes_name_every_kernel(plan):  # noqa: F811
    got = plan([(*size, which[2], 152) for which, size in VARIANTS.items()])
    for which, (P, S, rows, NT, MT, T, blocks, *_) in zip(VARIANTS, got):
        assert (P, int(S > 1), which[2], blocks) == which
    blocks = {1: (1, 2, 4, 6), 2: (4, 6)}
    assert set(VARIANTS) == {(P, s, g, b) for P in (1, 2) for s in (0, 1) for g in (0, 1) for b in blocks[P]}


def test_registers_are_allotted_in_units(tmp_path):
    """A kernel of 89 registers a thread is launched with as many as one of 96."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "r.cpp").write_text('#include <cstdio>\n#include "int8_plan.h"\n'
                                    "int main() { for (int n = 1; n < 103; ++n) std::putchar(sesg::int8_registers_fit(n) ? '1' : '0'); }\n")
    subprocess.run([cxx, "-std=c++17", "-I", f"{ROOT}/sparse_expert_swiglu_gb300/csrc", str(tmp_path / "r.cpp"), "-o",
                    str(tmp_path / "r")], check=True)
    out = subprocess.run([str(tmp_path / "r")], capture_output=True, text=True, check=True).stdout
    assert out == "0" * 88 + "1" * 14


@gpu
@pytest.mark.parametrize("which", VARIANTS)
def test_every_kernel(which):
    M, N, K = VARIANTS[which]
    for x, dtype, out, parts in (("int8", F16, F32, False), ("16 bits", BF16, None, True)):
        _linear_check(_linear_case(M, N, K, dtype, x, "silu" if which[2] else "gelu", parts, bool(which[2]), parts, out))
