"""Sizes that the C structures of the 8-bit operators and the norms cannot hold: the binding refuses them with ValueError, like every
other argument outside its range, before it makes a result."""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.test_int8 import F16, I8  # noqa: E402

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


@gpu
def test_more_tokens_than_32_bits_count():
    x = torch.empty(1 << 31, 16, dtype=F16, device="cuda")  # (not read)
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    w, ws = torch.zeros(1, 16, dtype=I8, device="cuda"), torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        ses.linear_int8(x, w, ws)
    for kw in (dict(), dict(int8=True), dict(norm="none"), dict(residual=x, residual_out=x)):
        with pytest.raises(ValueError):
            ses.residual_norm(x, **kw)
    assert torch.cuda.max_memory_allocated() < held + (1 << 20)  # no result of that size was made on the way
    del x
    torch.cuda.empty_cache()
