"""The plans of the calls on uncompressed weights, compiled by the host compiler alone: what a thread keeps, and what a
layer's workspace holds.  152 SMs and 227 KB of shared memory, as the GPU has."""

from __future__ import annotations

import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SHIM = r"""
#include "linear_plan.h"
#include "layer_plan.h"
using namespace sesg;
constexpr int kSms = 152, kRoom = 232448 - 1024 - 256;
static const LinearPlan& plan(const int* c, int room) {
  return linear_plan(c[0], c[1], c[2], c[3], c[4], c[5], c[6], kSms, room);
}
extern "C" {
// asks for n plans (M, N, K, gated, kn, plain, fp32 result) one after the other; how many of them are still kept then
int plans_kept(const int* c, int n) {
  const LinearPlan* at[1024];
  for (int i = 0; i < n; ++i) at[i] = &plan(c + 7 * i, kRoom);
  int kept = 0;
  for (int i = 0; i < n; ++i) {
    const int* q = c + 7 * i;
    kept += at[i]->M == q[0] && at[i]->N == q[1] && at[i]->K == q[2] && at[i]->gated == q[3] && at[i]->kn == q[4] &&
            at[i]->plain == q[5] && at[i]->f32 == q[6];
  }
  return kept;
}
// stages of the chosen tile for `room` bytes, after a call with `before` bytes
int stages_for(const int* c, int before, int room) {
  plan(c, before);
  bool own_x;
  const LinearPlan& l = plan(c, room);
  return linear_stages(l, c[0], c[3], room, own_x);
}
// an fp32 (16-bit) result's accumulators: the most chunks of 64 k that one takes, -1: without room in TMEM
int most_chunks(const int* c) {
  const LinearPlan& l = plan(c, kRoom);
  if (!l.S) return -1;
  const int KC = (c[2] + 63) / 64;
  if (l.by_token) return KC < sum_chunks(c[6]) ? KC : sum_chunks(c[6]);
  LinearSums s;
  if (!linear_sums(l, c[2], c[6], s) || s.cols > 512 || (s.keep && (l.both ? 2 : 1) * l.NT > 256)) return -1;
  return (s.per + s.groups - 1) / s.groups * l.wide;
}
size_t layer_bytes(int B, int d, int f, int E, int k, int ns) {
  return layer_plan(B, d, f, E, k, ns, kSms, 23 << 10, 4736).total;
}
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plans")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    csrc = os.path.join(ROOT, "sparse_expert_swiglu_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-fPIC", "-shared", "-I", csrc, str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def _ints(cases):
    flat = list(itertools.chain.from_iterable(cases))
    return (ctypes.c_int * len(flat))(*flat)


def _expert(n, d, f):
    """The two products of an expert on n tokens: gate and up with a split result or not, then down on pairs or not."""
    two = n <= 64
    return [(n, f, d, 1, 0, int(not two), 0), (2 * n if two else n, d, f, 0, 1, int(not two), 0)]


@pytest.mark.parametrize("d,f", [(5120, 8192), (4096, 14336), (2048, 1408), (6144, 16384), (4096, 4096), (8192, 8192)])
def test_both_products_of_an_expert_are_kept(plans, d, f):
    for n in list(range(1, 600, 7)) + [1024, 2048]:
        assert plans.plans_kept(_ints(_expert(n, d, f)), 2) == 2, n


def test_a_models_products_are_kept(plans):
    """One token count at a time: projections, dense block, output head and experts of a model."""
    for n in (1, 2, 3, 7, 16, 64, 65, 100, 256, 300, 512, 2048):
        for d, f, vocab in ((4096, 14336, 32000), (2048, 1408, 102400), (6144, 16384, 32768)):
            cases = [(n, d, d, 0, 0, 1, 0), (n, d + d // 4, d, 0, 0, 1, 0), (n, vocab, d, 0, 0, 1, 1), (n, f, d, 1, 0, 1, 0),
                     (n, d, f, 0, 1, 1, 0), (n, d, f, 0, 0, 1, 0), (n, 8, d, 0, 1, 1, 1), (n, 64, d, 0, 1, 1, 0)]
            cases += _expert(n, d, f)
            cases = list(dict.fromkeys(cases))
            assert plans.plans_kept(_ints(cases), len(cases)) == len(cases), (n, d)


def test_a_plan_goes_by_the_shared_memory_too(plans):
    """The same sizes with half the shared memory: the tile's stages fit."""
    case = _ints([(1024, 4095, 4096, 0, 0, 1, 0)])
    room = 232448 - 1024 - 256
    assert plans.stages_for(case, room, room) >= 2
    assert plans.stages_for(case, room, room // 4) >= 2


def test_no_accumulator_adds_up_more_than_its_share(plans):
    import random
    rng = random.Random(7)
    for _ in range(3000):
        size = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
        gated, kn, f32 = (rng.randint(0, 1) for _ in range(3))
        case = (size(1, 8192), 8 * size(1, 4096) if kn else size(1, 32768), 8 * size(1, 32768), gated, kn, 1, f32)
        most = plans.most_chunks(_ints([case]))
        assert 0 < most <= (16 if f32 else 256), (case, most)


# ---------------------------------------------------------------------------
# a layer's workspace
# ---------------------------------------------------------------------------

def _layer_bytes(plans, B, d, f, E, k, ns):
    plans.layer_bytes.restype = ctypes.c_size_t
    return plans.layer_bytes(B, d, f, E, k, ns)


@pytest.mark.parametrize("B,d,f,E,k,ns,mb", [(64, 2048, 1408, 64, 6, 2, 40), (64, 7168, 2048, 256, 8, 1, 100),
                                             (1, 4096, 14336, 8, 2, 0, 25), (17, 4096, 14336, 8, 2, 0, 25),
                                             (64, 16384, 65536, 256, 8, 8, 1000)])
def test_layer_workspace_bytes(plans, B, d, f, E, k, ns, mb):
    assert _layer_bytes(plans, B, d, f, E, k, ns) < mb * 1e6


def test_layer_workspace_holds_one_sum_a_pair_and_the_cut_tiles(plans):
    """Twice what cannot be done without (h of every token's experts as two rows in groups of 8, their fp32 sums, the
    logits), and 64 KB for each of at most 2 x 152 shares of cut tiles."""
    import random
    rng = random.Random(4)
    for _ in range(300):
        B, E = rng.randint(1, 64), rng.randint(1, 256)
        k, ns = rng.randint(1, min(8, E)), rng.randint(0, 8)
        d, f = 8 * rng.randint(1, 1024), 8 * rng.randint(1, 2048)
        pairs, active = B * k, min(E, B * k)
        groups = active + (pairs - active) // 8 + ns * ((B + 7) // 8)
        rows = 8 * groups if B <= 8 else pairs + B * ns
        need = groups * 16 * f * 2 + rows * d * 4 + B * 16 * E * 4 + B * d * 4
        assert _layer_bytes(plans, B, d, f, E, k, ns) <= 1.05 * need + 2 * 152 * 65536 + 65536, (B, d, f, E, k, ns)
