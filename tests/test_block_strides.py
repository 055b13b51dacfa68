"""Row strides that the block operators' C calls refuse: the last row of a
tensor has to lie within 63 bits of its first (no GPU needed)."""
import ctypes

import pytest

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import ufp4 as U

A = 0x10000                # an address that is never dereferenced
T, LD = 1 << 30, 1 << 40   # 2^30 rows, 2^40 elements apart: 2^70
MUCH = (1 << 63) - 1
SHAPE = -2


def routing():
    return (ctypes.c_void_p * 8)(*[A] * 8)


CALLS = {
    "norm, x": lambda L, d: L.ufp4_rmsnorm(A, LD, None, 0, A, d, d, T, 8, 1e-6, A, A, A, A, A, None),
    "norm, residual": lambda L, d: L.ufp4_rmsnorm(A, 8, A, LD, A, d, d, T, 8, 1e-6, A, A, A, A, A,
                                                  None),
    "norm_bwd, dy": lambda L, d: L.ufp4_rmsnorm_bwd(A, LD, A, 8, A, A, None, 0, d, d, T, 8, A, A, A,
                                                    MUCH, None),
    "norm_bwd, h": lambda L, d: L.ufp4_rmsnorm_bwd(A, 8, A, LD, A, A, None, 0, d, d, T, 8, A, A, A,
                                                   MUCH, None),
    "norm_bwd, dh": lambda L, d: L.ufp4_rmsnorm_bwd(A, 8, A, 8, A, A, A, LD, d, d, T, 8, A, A, A,
                                                    MUCH, None),
    "route": lambda L, d: L.ufp4_moe_route(A, LD, d, None, T, 8, 1, 1, routing(), A, MUCH, None),
    "route_bwd": lambda L, d: L.ufp4_moe_route_bwd(A, LD, d, T, 8, 1, 1, routing(), A, A, A, None),
    "dispatch": lambda L, d: L.ufp4_moe_dispatch(A, LD, A, d, T, 1, 8, A, None),
    "combine": lambda L, d: L.ufp4_moe_combine(A, A, A, A, LD, d, T, 1, 8, A, None),
    "combine_bwd": lambda L, d: L.ufp4_moe_combine_bwd(A, LD, A, A, A, d, T, 1, 8, A, A, None),
}


@pytest.mark.parametrize("dtype", [U.OUT_F32, U.OUT_BF16])
@pytest.mark.parametrize("call", CALLS)
def test_rows_past_63_bits_are_refused(call, dtype):
    assert CALLS[call](B.lib(), dtype) == SHAPE


def test_a_single_row_has_any_stride():
    """It is not used: the call goes on to refuse the missing pointer."""
    assert B.lib().ufp4_moe_dispatch(None, LD, A, U.OUT_F32, 1, 1, 8, A, None) == -1
    assert B.lib().ufp4_moe_dispatch(A, LD, A, U.OUT_F32, 0, 1, 8, A, None) == 0
