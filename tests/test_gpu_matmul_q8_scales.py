"""Activation scales far from one in the product of 8-bit activations with ternary
weights: a result that fits the output type is right, whatever the scales' sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import q8_util as R  # noqa: E402

tern = pytest.importorskip("ternary_weight_matmul_amd")

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def problem(M, N, K, group, seed, xs, ws):
    """Codes, packed weights, and scales log-uniform over the ranges xs and ws."""
    rng = np.random.default_rng(seed)
    q = rng.integers(-127, 128, (M, K)).astype(np.int8)
    x = np.exp(rng.uniform(*np.log(xs), (M, K // 128 if group else 1))).astype(np.float32)
    packed = rng.integers(0, 256, (N, K // 4)).astype(np.uint8)
    w = np.exp(rng.uniform(*np.log(ws), (N, K // 128))).astype(np.float16)
    return q, x, packed, w


def check(q, xs, packed, ws, what):
    print(f"{what}: M={q.shape[0]} N={packed.shape[0]} K={q.shape[1]} scales {xs.shape}", flush=True)
    want, bound = R.product(q, xs, packed, ws, torch.float32)
    assert (np.abs(want) < 3.4e38).all()
    # below 2^-126 every one of the sums' steps is off by up to half of the smallest number instead
    bound = bound + (ws.shape[1] + 8) * 2.0 ** -150
    y = tern.matmul_q8(dev(q), dev(xs), dev(packed), dev(ws), out_dtype=torch.float32)
    R.assert_close(y, want, bound, what)


# each of the kernels: up to 4 rows, few rows, tiles of 64 x 128 (K < 512 or more rows), tiles of 128 x 384
SIZES = [(1, 200, 640), (2, 130, 1152), (3, 33, 384), (4, 200, 640), (5, 64, 640), (16, 200, 640), (30, 100, 1152),
         (6, 200, 384), (33, 130, 640), (70, 200, 256), (600, 1000, 384), (1100, 7501, 2816)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group", [0, 128])
def test_large_scales(M, N, K, group):
    # a block's sum is at most 2^14: it leaves fp32 if it meets these before the weights' scale
    check(*problem(M, N, K, group, M + N, (1e35, 2e36), (1e-4, 5e-4)), "large scales")


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group", [0, 128])
def test_large_scales_of_both(M, N, K, group):
    """The product of both scales of a block leaves fp32, its sum is zero."""
    q, xs, packed, ws = problem(M, N, K, group, M + N, (1e34, 2e34), (1e-4, 1e-2))
    ws[:, 1] = 6e4
    q[:, 128:256] = 0
    check(q, xs, packed, ws, "large scales of both")


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group", [0, 128])
def test_small_scales(M, N, K, group):
    # products of two scales below fp32's normal range, sums on either side of its border
    check(*problem(M, N, K, group, M + N, (1e-42, 1e-37), (1e-5, 1e-3)), "small scales")


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group", [0, 128])
def test_results_next_to_the_largest_number(M, N, K, group):
    q, xs, packed, ws = problem(M, N, K, group, M + N, (1, 2), (1, 2))
    t = np.zeros((N, K), dtype=np.int64)
    t[np.arange(N), np.arange(N) % K] = np.where(np.arange(N) % 3 == 0, -1, 1)
    q[:] = 127
    xs[:] = 2.6e36      # 3.3e38
    ws[:] = 1
    check(q, xs, R.pack_ternary(t), ws, "large results")
