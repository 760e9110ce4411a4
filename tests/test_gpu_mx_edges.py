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
