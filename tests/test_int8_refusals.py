"""Calls of the 8-bit operators that the documentation rules out and that have to be refused before anything is enqueued."""

from __future__ import annotations

import pytest

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.test_int8 import ALIGN, INVALID, SMALL, X, _c_expert  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


@pytest.mark.parametrize("dtype", [0, 1])
def test_expert_output_in_a_part_of_its_tokens(dtype):
    """y may be x's buffer, not a part of it: tokens that the caller may still need would go."""
    nbytes = 2 * 64 * 2  # of x and of y
    ok = dict(x_dtype=dtype, dtype=dtype, xs=None)
    for at in (X - nbytes + 16, X - 128, X - 16, X + 16, X + 128, X + nbytes - 16):
        assert _c_expert(**ok, y=at) == INVALID, at - X
        assert _c_expert(**ok, y=at, residual=at) == INVALID, at - X
    for at in (X - nbytes, X, X + nbytes):
        assert _c_expert(**ok, y=at) == SMALL and _c_expert(**ok, y=at, residual=at) == SMALL
    assert _c_expert(**ok, y=X + 8) == ALIGN
