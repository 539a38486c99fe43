"""Sizes of MXFP4 matrices near their limits (no GPU: what is refused is
refused before anything is launched, and nothing else is called)."""
import ctypes

import pytest

from sparse_mixture_experts_renorm_b200 import MoEError, _binding as B, build as build_mod, mx_scale_bytes

P = ctypes.c_void_p(4096)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def test_scale_bytes_of_ragged_groups_count_the_rows_once(lib):
    """`rows` of a ragged matrix are those of all groups, so 256 groups of 2^23 rows in all are valid."""
    assert lib.moe_mx_scale_bytes(256, 1 << 23, 32, 1) == 2 * ((1 << 15) + 256) * 1024
    assert mx_scale_bytes(256, (1 << 31) - 1, 64, True) == 2 * ((1 << 23) - 1 + 256) * 1024
    assert lib.moe_mx_scale_bytes(256, 1 << 23, 32, 0) == 0
    for bad in ((0, 5, 32), (-1, 5, 32), (2, -1, 32), (2, 5, 0), (2, 5, 40)):
        assert lib.moe_mx_scale_bytes(*bad, 1) == 0 and B.last_error_detail(lib)
    with pytest.raises(MoEError):
        mx_scale_bytes(0, 5, 32, True)


@pytest.mark.parametrize("groups,rows", [(256, 1 << 23), (200, 1 << 24), (256, (1 << 31) - 1)])
def test_scales_without_room_are_refused_at_any_number_of_rows(lib, groups, rows):
    n = lib.moe_mx_scale_bytes(groups, rows, 32, 1)
    for have in (0, 4096, n - 1):
        assert lib.moe_mx_quantize(P, P, groups, rows, 32, B.MOE_BF16, P, P, have, None) == B.MOE_ERR_INVALID_ARG
        assert lib.moe_mx_dequantize(P, P, have, P, groups, rows, 32, B.MOE_BF16, P, None) == B.MOE_ERR_INVALID_ARG
        assert str(n) in B.last_error_detail(lib)


def test_the_longest_row(lib):
    cols = (1 << 31) - 32
    assert lib.moe_mx_scale_bytes(1, 1, cols, 0) == 2 * 1024 * (1 << 23) == lib.moe_mx_scale_bytes(1, 1, cols, 1)
    n = lib.moe_mx_scale_bytes(1, 1, cols, 0)
    assert lib.moe_mx_quantize(P, None, 1, 1, cols, B.MOE_BF16, P, P, n - 1, None) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("offsets,groups,M,N", [(None, 1, 8, (1 << 31) - 8), (None, 1, (1 << 31) - 100, 8), (P, 3, (1 << 31) - 255, 8),
                                                (None, 2, 8, (1 << 30) - 8), (None, 5, 429496729, 8)])
def test_products_whose_last_tile_would_end_past_2_31_are_refused(lib, offsets, groups, M, N):
    """A tile's last row and column are 32-bit numbers: past them a column would compare as a negative one."""
    st = lib.moe_mx_matmul(P, P, P, P, offsets, groups, M, N, 32, B.MOE_F32, P, P, None)
    assert st == B.MOE_ERR_UNSUPPORTED and "too large" in B.last_error_detail(lib)


@pytest.mark.parametrize("T,E,I", [(1, 62, 34636832), (((1 << 31) - 256) // 8 + 8, 8, 32)])
def test_experts_whose_last_tile_would_end_past_2_31_are_refused(lib, T, E, I):
    assert lib.moe_mx_workspace_size(T, 32, E, 8, I) == 0 and B.last_error_detail(lib)
