"""Largest stacks of the orthogonalisation: refused before anything is launched, or held by every launch (no GPU is touched)."""
import ctypes

import pytest

import mixture_experts_expert_histogram_amd as moe
from mixture_experts_expert_histogram_amd import _lib
from tests.test_block_abi import BIG, ORTHO, P, call, ortho_desc


# with a side below 64 the update runs on tiles of at most 128 x 128: 2^24 of these are 2^32 threads
@pytest.mark.parametrize("E,M,N", [(32768, 8, 1 << 16), (2048, 8, 1 << 20), (2048, 1 << 20, 8), (1100, 56, 1 << 20), (65535, 1 << 15, 40)])
def test_narrow_stacks_of_more_tiles_than_a_launch_holds(E, M, N):
    d = ortho_desc(E=E, M=M, N=N)
    assert call(ORTHO[0], d, ORTHO[1], {}) == _lib.MOE_ERR_UNSUPPORTED
    opt = _lib.Muon(0.1, 0.9, 0.0, 1)
    assert moe.library().moe_muon_step(ctypes.byref(d), ctypes.byref(opt), *[P] * 6, BIG, None) == _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("E,M,N", [(1024, 8, 1 << 20), (16384, 1 << 16, 56), (2048, 64, 1 << 20), (2048, 1 << 20, 256)])
def test_largest_stacks_that_are_taken(E, M, N):
    assert moe.ortho_workspace_size(ortho_desc(E=E, M=M, N=N)) > 0
