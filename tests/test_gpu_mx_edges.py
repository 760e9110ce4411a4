"""Products with microscaled weights at the ends of the types: infinities and
NaN, scales over the whole range of the exponent byte, activations that need
all their bits, and the largest sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mx_util as R  # noqa: E402
from test_gpu_mx import DEV, DT, _need_gpu, activations, dev, nan_out, weights  # noqa: E402,F401

tern = pytest.importorskip("ternary_weight_matmul_amd")

# one shape for each kernel and tile: few rows, sixteens of rows, small tiles, big tiles
PLACES = [(1, 40, 288), (4, 72, 1056), (16, 40, 512), (70, 300, 288), (200, 130, 1056), (700, 9300, 96)]


@pytest.mark.parametrize("M,N,K", PLACES)
@pytest.mark.parametrize("xd", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [{"f16": 0x7C00, "bf16": 0x7F80}, {"f16": 0xFC00, "bf16": 0xFF80},
                                  {"f16": 0x7C01, "bf16": 0x7F81}, {"f16": 0xFE00, "bf16": 0xFFC0}],
                         ids=["inf", "-inf", "nan1", "nan"])
def test_infinities_and_nan_follow_the_sum(M, N, K, xd, bits):
    """An infinity times a weight is an infinity of the product's sign, times 0 a NaN; a NaN
    reaches its whole row."""
    print(f"{M}x{K}->{N} {xd} {bits[xd]:x}", flush=True)
    codes, exps = weights(N, K, 31)
    x = activations(M, K, xd, 32)
    clean = tern.mx_matmul(x.to(DEV), dev(codes), dev(exps), out_dtype=torch.float32)
    m, k = M // 2, K // 3
    x.view(torch.int16)[m, k] = int(np.array(bits[xd], dtype=np.uint16).view(np.int16))
    y = tern.mx_matmul_into(x.to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    w = R.values(codes, exps)[:, k]
    with np.errstate(invalid="ignore"):
        want = (R.f64(x)[m, k] * w).astype(np.float32)
    assert np.array_equal(y[m].cpu().numpy(), want, equal_nan=True)
    keep = [i for i in range(M) if i != m]
    assert torch.equal(y[keep], clean[keep])


@pytest.fixture
def free_memory():
    """Nothing cached before a test that takes most of the memory, nor left behind it."""
    torch.cuda.empty_cache()
    yield torch.cuda.mem_get_info()[0]
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N,kind", [(2 ** 31 - 1, 1, "mx"), (2 ** 31 - 300, 2, "mx"), (33, 2 ** 31 - 1, "bf16"),
                                      (60, 2 ** 30 - 4, "bf16")])
def test_most_rows_and_columns(M, N, kind, free_memory):
    """Sizes whose tiles would be too many threads for a launch, or have columns past 2^31; the sums
    are exact, and the rows and columns that differ are the last ones and some in between."""
    K = 32
    need = (M + N) * 17 * (4 if kind == "bf16" and M > N else 1) + 2 * M * N + (8 << 30)
    if free_memory < need:
        pytest.skip(f"needs {need >> 30} GB")
    print(f"{M}x{K}->{N} {kind}, {need >> 30} GB", flush=True)
    codes = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device=DEV)   # ones
    exps = torch.full((N, 1), 127, dtype=torch.uint8, device=DEV)
    cols = sorted({0, N // 3, max(N - 130, 0), max(N - 2, 0), N - 1})
    rows = sorted({0, M // 3, max(M - 300, 0), max(M - 2, 0), M - 1})
    for i, c in enumerate(cols):
        codes[c] = 0
        codes[c, i] = 0x40                                                 # a two at 2 i + 1
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    if kind == "mx":
        xc = torch.full((M, K // 2), 0x11, dtype=torch.uint8, device=DEV)  # halves
        xe = torch.full((M, 1), 127, dtype=torch.uint8, device=DEV)
        for i, r in enumerate(rows):
            xc[r, 1:] = 0
            xc[r, 0] = 0x51                                                # a half and a three
        tern.mx_matmul_mx_into(xc, xe, codes, exps, y)
    else:
        x = torch.full((M, K), 0.5, dtype=torch.bfloat16, device=DEV)
        for i, r in enumerate(rows):
            x[r, 2:] = 0
            x[r, 1] = 3.0
        tern.mx_matmul_into(x, codes, exps, y)

    def want(m, n):
        row = [0.5, 3.0] + [0.0] * 30 if m in rows else [0.5] * 32
        return 2 * row[2 * cols.index(n) + 1] if n in cols else sum(row)

    for r in rows + [1, M // 2]:
        for c in cols + [min(1, N - 1), N // 2]:
            assert float(y[r, c]) == want(r, c), (r, c)
    # everything else is one value
    flat, step, other = y.view(-1), 1 << 30, 0
    for at in range(0, flat.numel(), step):
        other += int((flat[at:at + step] != 16).sum())
    assert other == M * N - (M - len(rows)) * (N - len(cols))


@pytest.mark.parametrize("M,N,K", [(1, 24, 288), (2, 72, 1056), (4, 100, 512), (8, 40, 1184), (16, 130, 544),
                                   (24, 33, 320), (70, 300, 288), (200, 130, 1056), (700, 9300, 96)])
def test_every_bit_of_fp16_activations(M, N, K):
    """Integers of 11 significant bits in every place, against multiples of a half: all sums are
    exact, so an activation's last bits are seen wherever they are lost or misplaced."""
    rng = np.random.default_rng(M + N)
    x = rng.integers(1025, 2048, (M, K)) * rng.choice([-1.0, 1.0], (M, K))
    x[rng.random((M, K)) < 0.5] *= 0.5   # two exponents side by side, sums are multiples of a quarter
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    exps = np.full((N, K // 32), 127, dtype=np.uint8)
    W = R.values(codes, exps)
    assert (np.abs(x) @ np.abs(W).T).max() * 4 < 2 ** 24
    want = x @ W.T
    xt = torch.from_numpy(x).half()
    assert np.array_equal(R.f64(xt), x)
    y = tern.mx_matmul_into(xt.to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    assert np.array_equal(R.f64(y), want)


@pytest.mark.parametrize("M", [1, 4, 9, 255])
def test_every_pair_of_scales_of_4_bit_operands(M):
    """One value in a block of zeros: the product's scale is the sum of two exponent bytes, over all
    255 x 255 of them, subnormal results and infinities included."""
    K, k, rows = 96, 40, torch.arange(255, dtype=torch.uint8)
    wc = torch.full((255, K // 2), 0x22, dtype=torch.uint8)   # ones
    we = rows[:, None].repeat(1, K // 32)
    for a in range(0, 255, M):
        xe = rows[a:a + M, None].repeat(1, K // 32)
        xc = torch.zeros((xe.shape[0], K // 2), dtype=torch.uint8)
        xc[:, k // 2] = 2
        y = tern.mx_matmul_mx(xc.to(DEV), xe.to(DEV), wc.to(DEV), we.to(DEV), out_dtype=torch.float32).cpu()
        want = torch.pow(2.0, (xe[:, :1].double() - 127) + (rows[None].double() - 127)).float()
        assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [(1, 40, 1056), (6, 130, 288), (16, 64, 512), (70, 300, 288), (300, 600, 544)])
def test_4_bit_operands_with_scales_far_apart(M, N, K):
    """Blocks whose scales differ by up to 2^60, zero blocks (exponent 0) among them: within the bound
    of fp32 sums of exact products."""
    rng = np.random.default_rng(K)
    xc, wc = (rng.integers(0, 256, (r, K // 2)).astype(np.uint8) for r in (M, N))
    xe, we = (rng.integers(97, 158, (r, K // 32)).astype(np.uint8) for r in (M, N))
    zero = rng.random((M, K // 32)) < 0.2
    zero[:, 0] = True
    xe[zero] = 0
    xc.reshape(M, K // 32, 16)[zero] = 0
    X, W = R.values(xc, xe), R.values(wc, we)
    want = X @ W.T
    y = tern.mx_matmul_mx_into(dev(xc), dev(xe), dev(wc), dev(we), nan_out(M, N, "f32"))
    R.assert_close(y, want, R.product_bound(X, W, want, torch.float32))


@pytest.mark.parametrize("M,N,K", [(1, 255, 64), (5, 255, 1056), (70, 255, 288), (300, 600, 544)])
@pytest.mark.parametrize("xd", ["f16", "bf16"])
@pytest.mark.parametrize("v", [1.0, 2.0 ** -14, 3 * 2.0 ** 12])
def test_every_scale_against_16_bit_activations(M, N, K, xd, v):
    """Single weights of a half read back through every exponent byte but 255, subnormal bf16 weights
    and subnormal results included."""
    exps = np.repeat((np.arange(N) % 255).astype(np.uint8)[:, None], K // 32, axis=1)
    codes = np.full((N, K // 2), 0x11, dtype=np.uint8)
    x = torch.zeros((M, K))
    x[torch.arange(M), (torch.arange(M) * 37 + 5) % K] = v
    y = tern.mx_matmul_into(x.to(DT[xd]).to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32")).cpu()
    with np.errstate(over="ignore"):
        want = (0.5 * v * np.exp2(exps[:, 0].astype(np.float64) - 127)).astype(np.float32)
    assert np.array_equal(y.numpy(), np.broadcast_to(want, (M, N)))


@pytest.mark.parametrize("M,N,K", [(200, 64, 5120), (1024, 16, 17408), (161, 1, 96), (2048, 8, 1056), (176, 1024, 288),
                                   (177, 1489, 160), (513, 496, 544)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "mx"])
def test_many_rows_by_a_narrow_matrix(M, N, K, kind):
    """The products of a router over a prompt, on either side of the border between the kernels."""
    print(f"{M}x{K}->{N} {kind}", flush=True)
    codes, exps = weights(N, K, M + N)
    if kind == "mx":
        xc, xe = weights(M, K, M * 3 + N, spread=4)
        X = R.values(xc, xe)
        y = tern.mx_matmul_mx_into(dev(xc), dev(xe), dev(codes), dev(exps), nan_out(M, N, "f32"))
    else:
        x = activations(M, K, kind, M)
        X = R.f64(x)
        y = tern.mx_matmul_into(x.to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    W = R.values(codes, exps)
    want = X @ W.T
    R.assert_close(y, want, R.product_bound(X, W, want, torch.float32))
