"""The number of tokens up to which linear attention counts rows in an int (refused before a launch,
so the fake pointers are never read)."""

import ctypes

import pytest

import gated_delta_rule_144_b200 as kda
from gated_delta_rule_144_b200 import build as kbuild


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


@pytest.mark.parametrize("B,T", [(1, (1 << 30) + 1), (1, (1 << 31) - 1), (3, 1 << 29)])
def test_too_many_tokens(L, B, T):
    """Segments are at least 1/148 of a long row, so that a segment's end passes 2^31 for rows
    this side of it already."""
    far = lambda i: ctypes.c_void_p(0x100000 + (i << 48))  # noqa: E731
    for dtype in (kda.KDA_BF16, kda.KDA_F32):
        d = kda.LinearDesc(B, T, 1, 1, 8, 8, B, dtype, 0)
        st = L.kda_linear_fwd(ctypes.byref(d), far(0), far(1), far(2), far(3), None, None, far(4),
                              None, far(5), 1 << 40, None)
        assert st == 1 and b"too large" in L.kda_last_error()
        assert L.kda_linear_fwd_workspace_size(ctypes.byref(d)) == 0
        st = L.kda_linear_decode(B, T, 1, 1, 8, 8, dtype, 0, far(0), far(1), far(2), far(3), far(6),
                                 far(4), None)
        assert st == 1 and b"too large" in L.kda_last_error()


def test_the_most_tokens_have_a_plan(L):
    n = kda.linear_fwd_workspace_size
    import torch
    for dtype in (torch.bfloat16, torch.float32):
        assert 0 < n(1, 1 << 30, 1, 1, 8, 8, 1, dtype) < 1 << 36
