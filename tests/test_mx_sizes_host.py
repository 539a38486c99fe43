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
