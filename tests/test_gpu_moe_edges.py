"""The mixture-of-experts layer where a token's result could depend on its
companions or on the kernel that its batch takes: scales that are not finite,
precision and range of the hidden values."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mx_util as R  # noqa: E402
from test_gpu_moe import DEV, Layer, _need_gpu, inputs  # noqa: E402,F401  (the fixture skips without a GPU)

tern = pytest.importorskip("ternary_weight_matmul_amd")


@pytest.mark.parametrize("T", [2, 3, 4, 5, 20, 70])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("where", ["down", "gate_up"])
@pytest.mark.parametrize("yd", ["bf16", "f32"])
def test_scales_stay_with_the_tokens_that_take_the_expert(T, bad, where, yd):
    """Only token 0 takes expert 5, whose scales are not finite: it gets what they make of its
    sum, the other tokens the bits that they get beside a finite expert, and a token that takes
    none gets zeros."""
    E, H, F, k = 6, 256, 640, 2
    print(f"T={T} {bad} in {where} {yd}", flush=True)
    L = Layer(E, H, F, 21, zeros=0.1)
    x, lg = inputs(T, E, H, "bf16", 22)
    lg[:, 5] = -10.0
    lg[0, 5] = 10.0
    lg[T - 1] = -float("inf")
    clean = L.run(x, lg, k, yd=yd)
    assert torch.isfinite(clean).all() and (clean[T - 1] == 0).all()
    scales = L.ds if where == "down" else L.gus
    scales[5] = bad
    L.d = None
    y = L.run(x, lg, k, yd=yd)
    assert torch.equal(y[1:], clean[1:])
    assert not torch.isfinite(y[0]).any()
