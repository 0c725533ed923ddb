"""Threads, CTAs and the form of the norms around a block, compiled as host code: what the kernel needs of them over the whole
range of sizes, and the sides of the border between its two forms that were measured.  On the GPU, both forms' bits."""

from __future__ import annotations

import random
import shutil
import subprocess

import pytest
import torch

from tests.conftest import ROOT

gpu = pytest.mark.gpu

SOURCE = r"""
#include <cstdio>
#include "norm_plan.h"
using namespace sesg;
int main() {
  int M, d, residual, s_f32, y_int8, sms;
  while (std::scanf("%d %d %d %d %d %d", &M, &d, &residual, &s_f32, &y_int8, &sms) == 6) {
    const NormPlan l = norm_plan(M, d, residual, s_f32, y_int8, sms);
    std::printf("%d %d %d %d %d\n", (int)l.ahead, l.nv, l.threads, l.ctas, (int)l.bytes);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plans")
    (d / "p.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", f"{ROOT}/sparse_expert_swiglu_gb300/csrc", str(d / "p.cpp"), "-o", str(d / "p")],
                   check=True)

    def run(sizes):
        text = "".join("%d %d %d %d %d %d\n" % s for s in sizes)
        out = subprocess.run([str(d / "p")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_what_the_kernel_needs(plan):
    r = random.Random(6)
    sizes = [(M, d, a, b, c, sms) for M in (1, 152, 305, 1 << 20) for d in (8, 512, 520, 4096, 8192, 8200, 16384)
             for a in (0, 1) for b in (0, 1) for c in (0, 1) for sms in (152, 148, 1)]
    sizes += [(int(2 ** r.uniform(0, 20)), 8 * int(2 ** r.uniform(0, 11)), r.randint(0, 1), r.randint(0, 1), r.randint(0, 1),
               r.choice((152, 148, 16))) for _ in range(3000)]
    for (M, d, residual, s_f32, y_int8, sms), (ahead, nv, threads, ctas, nbytes) in zip(sizes, plan(sizes)):
        what = (M, d, residual, s_f32, y_int8, sms)
        # every vector of 8 has a thread, whole warps
        assert nv in (1, 2) and threads % 32 == 0 and 32 <= threads <= 1024 and nv * threads * 8 >= d, what
        assert 1 <= ctas <= M, what
        if ahead:  # only this form goes on to further tokens
            assert nv == 2 and nbytes == 2 * (1 if not residual else 3 if s_f32 else 2) * threads * 16 and nbytes <= 200 << 10, what
        else:
            assert ctas == M and nbytes == 0, what


def test_the_measured_border(plan):
    """No copies ahead where they only delay: one token for each CTA, of few values each."""
    plain = [(305, 512, 1, 0, 1), (608, 512, 1, 1, 0), (608, 1024, 1, 0, 0), (400, 1024, 1, 1, 0), (608, 2048, 1, 0, 1), (608, 2048, 1, 1, 0),
             (2553, 256, 1, 0, 0), (5836, 256, 1, 0, 1), (305, 64, 0, 0, 0), (304, 8192, 1, 0, 0), (1, 16384, 0, 0, 0)]
    ahead = [(305, 6144, 1, 0, 0), (400, 4096, 1, 0, 0), (608, 4096, 1, 1, 0), (851, 2048, 1, 0, 0), (1702, 1024, 1, 0, 0),
             (4742, 256, 1, 0, 0), (10944, 512, 1, 0, 1), (8192, 4096, 1, 1, 0), (1000, 8208, 1, 0, 1)]
    got = plan([(*s, 152) for s in plain + ahead])
    assert [g[0] for g in got] == [0] * len(plain) + [1] * len(ahead)


@gpu
@pytest.mark.parametrize("d", [264, 512, 1040, 2048])
def test_both_forms_give_the_same_bits(d):
    ses = pytest.importorskip("sparse_expert_swiglu_gb300")
    ses.build_library()
    from tests.test_residual_norm import BF16, _case, _cuda, _run
    for wide, int8, norm in ((False, False, "rms"), (True, False, "layer"), (False, True, "rms")):
        M = 12000
        a = {k: _cuda(v) for k, v in _case(M, d, BF16, "rms", norm, wide=wide, int8=int8 and d % 16 == 0).items()}
        full = _run(a)
        for first, n in ((0, 300), (M // 2, 610), (M - 2000, 2000)):
            rows = slice(first, first + n)
            some = _run({**a, "x": a["x"][rows], "residual": a["residual"][rows]})
            assert all(torch.equal(f[rows], s) for f, s in zip(full, some))
