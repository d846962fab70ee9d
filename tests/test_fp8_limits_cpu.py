"""Size limits of the block-scaled e4m3 functions at the C-ABI; no GPU."""
import ctypes
import os

import pytest

import int8_mixed_precision_outlier_amd as i8

FAKE = ctypes.c_void_p(1 << 20)  # aligned non-null; never dereferenced (checks fail first)
EINVAL, OK = i8.STATUS_EINVAL, i8.STATUS_OK

pytestmark = pytest.mark.skipif(not os.path.exists(i8.LIB_PATH),
                                reason="libint8mm.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("N", [(1 << 24) + 16, 1 << 27, (1 << 31) - 16, 1 << 31])
def test_features_without_columns(N):
    """K = 0 leaves N * roundup(K, 128) at 0 for every N: N has the bound that
    K = 16 gives it, so that it fits the kernels' integers and grids."""
    lib = i8.load()
    assert lib.fp8_packed_size(N, 0) == -1
    assert lib.fp8_matmul_config(1, N, 0, (ctypes.c_int32 * 4)()) == EINVAL
    assert lib.fp8_quantize_weight(FAKE, 0, 0, N, FAKE, FAKE, None) == EINVAL
    assert lib.fp8_pack_weight(FAKE, N, 0, FAKE, None) == EINVAL
    # no rows: nothing would be launched, whatever the check says
    assert lib.fp8_matmul(None, None, 0, 0, None, None, N, None, 0, FAKE, None) == EINVAL


def test_most_features_without_columns():
    lib = i8.load()
    N = 1 << 24
    assert lib.fp8_packed_size(N, 0) == 0
    assert lib.fp8_packed_size(N, 16) == lib.fp8_packed_size(N, 128) == N * 128
    assert lib.fp8_packed_size(N, 144) == -1
    cfg = (ctypes.c_int32 * 4)()
    for M in (1, 128):  # M * N = 2^31
        assert lib.fp8_matmul_config(M, N, 0, cfg) == OK
    assert lib.fp8_matmul_config(144, N, 0, cfg) == EINVAL
    assert lib.fp8_matmul(None, None, 0, 0, None, None, N, None, 0, FAKE, None) == OK
