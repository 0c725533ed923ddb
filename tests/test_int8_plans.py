"""The plans of the 8-bit products' tensor-core kernels, compiled as host code: what the kernel's barriers and memory need
of them, over the whole range of sizes."""

from __future__ import annotations

import random
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "int8_plan.h"
using namespace sesg;
int main() {
  int M, N, K, g, sms;
  while (std::scanf("%d %d %d %d %d", &M, &N, &K, &g, &sms) == 5) {
    const int room = 227 * 1024 - 1024 - 768 - int8_extra_bytes(g);
    const Int8Plan l = int8_plan(M, N, K, g, sms, room);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d %d\n", l.P, l.S, l.rows, l.NT, l.MT, l.T, l.blocks, l.stages, l.slots,
                int8_stage_bytes(l), int8_sum_bytes(l), room);
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
        text = "".join("%d %d %d %d %d\n" % s for s in sizes)
        out = subprocess.run([str(d / "p")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def _sizes():
    r = random.Random(4)
    some = [(M, N, K, g, sms) for M in (1, 9, 16, 17, 33, 64, 97, 300, 2048, 1 << 20) for N in (1, 64, 129, 1031, 4096, 1 << 20)
            for K in (16, 1008, 4096, 65536) for g in (0, 1) for sms in (152, 148)]
    for _ in range(2000):
        some.append((int(2 ** r.uniform(0, 14)), int(2 ** r.uniform(0, 17)), int(2 ** r.uniform(0, 12.0)) * 16, r.randint(0, 1),
                     r.choice((152, 148, 16))))
    return some


def test_plans_hold_what_the_kernel_needs(plan):
    sizes = _sizes()
    plans = plan(sizes)
    assert len(plans) == len(sizes)
    for (M, N, K, g, sms), (P, S, rows, NT, MT, T, blocks, stages, slots, stage, sums, room) in zip(sizes, plans):
        what = (M, N, K, g, sms, P, S, rows, NT)
        feats = 64 if g else 128
        assert P in (1, 2) and S in (1, 2, 4, 8) and P * S <= 8, what
        # two sets of warps take the stages by turns: a stage is always the same set's
        assert 2 <= stages <= 8 and stages % 2 == 0 and stages * stage <= room, what
        # 16 columns at least for each CTA's half of the tokens, whole 1024-byte groups of 8 rows
        assert NT % 16 == 0 and 16 <= NT <= 192 and (P == 1 or NT % 32 == 0), what
        assert MT * NT >= M and 1 <= rows <= feats and rows % 8 == 0, what
        assert T == -(-N // (rows * P)) * MT and T >= 1, what
        assert 32 * blocks >= NT and blocks in (1, 2, 4, 6) and (P == 1 or blocks >= 4), what
        # TMEM: two sets of accumulators and the slots; up to 64 tokens a slot is free when its stage is
        assert 2 * NT + slots * (32 if blocks == 6 else 64) <= 512 and 2 <= slots <= 8, what
        if blocks <= 2:
            assert slots >= stages, what
        else:
            # a slot's use before its last one ends before these warps' last wait: four stages back
            assert slots >= 4, what
        if S > 1:
            assert T * S * P <= sms and sums <= stages * stage and S <= -(-K // 128), what
