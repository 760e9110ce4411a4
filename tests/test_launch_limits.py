"""Numbers of threads of a launch: the kernels that a size is left to have fewer than 2^32."""
import ctypes

import pytest

pytest.importorskip("torch")
tern = pytest.importorskip("ternary_weight_matmul_amd", reason="libtern.so not built")

BF16, CODES = 1, 3


def fits(M, N, K, x_dtype):
    """bool tern::gemv_fp4_fits(int64_t, int64_t, int64_t, int): whether the decode kernel takes a product."""
    f = ctypes.CDLL(tern.library_path())["_ZN4tern13gemv_fp4_fitsEllli"]
    f.argtypes, f.restype = [ctypes.c_int64] * 3 + [ctypes.c_int], ctypes.c_bool
    return f(M, N, K, x_dtype)


@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("x_dtype", [BF16, CODES])
def test_decode_kernel_takes_what_a_launch_holds(M, x_dtype):
    for N, K in ((1, 128), (5120, 5120), (17408, 5120), (5120, 17408), (1 << 20, 8192), (1 << 24, 5120)):
        assert fits(M, N, K, x_dtype)
    # 64 * 16 threads for at most 17 quads of 4 rows
    assert not fits(M, 1 << 30, 8192, x_dtype)
    if M == 1:   # for 10 quads: 25.6 a row, 2^32 at 167.8 million rows
        assert fits(M, 160_000_000, 8192, x_dtype) and not fits(M, 170_000_000, 8192, x_dtype)
