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


@pytest.mark.parametrize("M,N,kind", [(2 ** 31 - 1, 1, "mx"), (2 ** 31 - 300, 2, "mx"), (33, 2 ** 31 - 1, "bf16"),
                                      (60, 2 ** 30 - 4, "bf16")])
def test_most_rows_and_columns(M, N, kind):
    """Sizes whose tiles would be too many threads for a launch, or have columns past 2^31; the sums
    are exact, and the rows and columns that differ are the last ones and some in between."""
    K = 32
    need = (M + N) * 17 * (4 if kind == "bf16" and M > N else 1) + 2 * M * N + (8 << 30)
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < need:
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
