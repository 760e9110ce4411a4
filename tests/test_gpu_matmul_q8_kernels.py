"""Every form of the kernels of the product of 8-bit activations: the numbers of weight rows,
of steps and of tiles by which they are chosen."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import q8_util as R  # noqa: E402
from test_gpu_matmul_q8 import problem, run  # noqa: E402

tern = pytest.importorskip("ternary_weight_matmul_amd")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(M, N, K, group, yd="f32"):
    print(f"matmul_q8 M={M} N={N} K={K} group={group} -> {yd}", flush=True)
    q, xs, packed, ws = problem(M, N, K, group, M + N + K, lo=-128)
    y = run(q, xs, packed, ws, yd)
    # some rows in full, and all rows of some columns
    cols = np.unique(np.concatenate([np.arange(0, N, max(1, N // 97)), np.arange(max(0, N - 40), N)]))
    rows = np.unique(np.r_[0, M // 2, M - 1])
    want, bound = R.product(q, xs, packed[cols], ws[cols], torch.float32 if yd == "f32" else torch.bfloat16)
    R.assert_close(y[:, torch.from_numpy(cols).to(y.device)], want, bound, "columns")
    want, bound = R.product(q[rows], xs[rows], packed, ws, torch.float32 if yd == "f32" else torch.bfloat16)
    R.assert_close(y[torch.from_numpy(rows).to(y.device)], want, bound, "rows")


# few rows: 1 to 5 sixteens of weight rows to a workgroup, with one and two sixteens of rows of X
@pytest.mark.parametrize("N", [4090, 4500, 5120, 8203, 12300, 16400, 17408])
@pytest.mark.parametrize("M", [5, 16, 17, 32])
@pytest.mark.parametrize("group", [0, 128])
def test_few_rows(M, N, group):
    check(M, N, 640, group)


# long K: codes for more turns ahead
@pytest.mark.parametrize("M", [5, 16, 20, 32])
@pytest.mark.parametrize("K", [12416, 17408])
@pytest.mark.parametrize("group", [0, 128])
def test_few_rows_with_long_k(M, K, group):
    check(M, 4200, K, group, "bf16")


# up to 4 rows: one to four steps a wave, and K beyond what its waves take
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("K", [8192, 12288, 20480, 28672, 32768, 33280, 65536])
@pytest.mark.parametrize("group", [0, 128])
def test_up_to_four_rows_with_long_k(M, K, group):
    check(M, 50, K, group)


# up to 4 rows: every number of weight rows of a workgroup
@pytest.mark.parametrize("M", [1, 4])
@pytest.mark.parametrize("N", [1000, 2000, 3000, 4000, 6000, 8000, 10000, 17408, 34816])
@pytest.mark.parametrize("group", [0, 128])
def test_up_to_four_rows(M, N, group):
    check(M, N, 640, group)


# tiles whose number is a multiple of 8 go round the dies in another order; more than one band of tile rows
@pytest.mark.parametrize("M,N,K", [(1100, 9001, 2816), (1024, 3000, 384), (1600, 1500, 256)])
@pytest.mark.parametrize("group", [0, 128])
def test_tiles_in_runs(M, N, K, group):
    assert (tern.lib.tern_matmul_q8_workspace(M, N, K) > 0) == (K == 2816)
    check(M, N, K, group, "bf16")


# large tiles with fewer blocks of K than they have buffers: one, two, three
@pytest.mark.parametrize("M,N,K", [(30700, 26877, 128), (20000, 26877, 256), (16300, 19197, 384)])
@pytest.mark.parametrize("group", [0, 128])
def test_large_tiles_of_few_blocks(M, N, K, group):
    assert tern.lib.tern_matmul_q8_workspace(M, N, K) > 0
    check(M, N, K, group, "bf16")
