"""Sizes of the weight gradient from 8-bit rows that the kernels cannot count, refused with no GPU touched."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

P = 0x10000  # 16-byte aligned non-null address; never dereferenced on these paths
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not real")


def wgrad(E, hidden, n, T=128):
    return kgw.load_library().kgw_wgrad_fp8_rows(P, P, P, None, P, E, hidden, n, T, None, P, 0, 0, None, 0, None)


# Tiles are counted in 32 bits, in whatever edge they have: 65536 experts of 64 x n take tiles of 128 there, twice as many as
# tiles of 256 (all but a few experts' outputs may be skipped, so the sizes need no memory).
@pytest.mark.parametrize("hidden,n", [(64, 1 << 22), (64, (1 << 23) - 1024), (128, 5 << 20), (8, 6 << 20)])
def test_more_tiles_than_are_counted(hidden, n):
    assert ((hidden + 255) // 256) * ((n + 255) // 256) * 65536 < 2 ** 31 - 1
    assert wgrad(65536, hidden, n) == kgw.KGW_ERROR_UNSUPPORTED


@no_gpu
@pytest.mark.parametrize("E,hidden,n", [(65536, 64, (1 << 22) - 128), (65536, 256, 1 << 22), (32768, 64, (1 << 23) - 256), (1, 64, 1 << 20)])
def test_as_many_as_are_counted(E, hidden, n):
    assert wgrad(E, hidden, n) == kgw.KGW_ERROR_DEVICE       # past the refusals
