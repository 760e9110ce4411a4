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


class Exact:
    """A layer whose every step is exact: one expert per token (weight 1), a gate of 256 (silu is
    the identity there), up rows that add a few of a token's integers with a scale of 1."""

    def __init__(self, E, H, F):
        self.L = Layer(E, H, F, 1)
        self.up = np.zeros((E, F, H), dtype=np.int64)
        self.down = np.zeros((E, H, F), dtype=np.int64)
        self.x = None

    def run(self, x, xd, yd, scale):
        L, T = self.L, x.shape[0]
        gate = np.zeros_like(self.up)
        gate[:, :, 0] = 1
        L.gu = R.pack_ternary(np.concatenate([gate, self.up], axis=1))
        L.dn = R.pack_ternary(self.down)
        L.gus = np.ones((L.E, 2 * L.F, L.H // 128), dtype=np.float16)
        L.ds = np.full((L.E, L.H, L.F // 128), scale, dtype=np.float16)
        x = x.copy()
        x[:, 0] = 256
        t = torch.from_numpy(x).to(xd)
        assert np.array_equal(R.f64(t), x)
        lg = torch.full((T, L.E), -1.0)
        chosen = np.arange(T) % L.E
        lg[torch.arange(T), torch.from_numpy(chosen)] = 1.0
        y = L.run(t, lg, 1, yd=yd)
        want = np.zeros((T, L.H))
        for i, e in enumerate(chosen):
            want[i] = (256 * (x[i] @ self.up[e].T)) @ self.down[e].T * scale
        return y, want


BATCHES = [1, 2, 3, 4, 5, 20, 70]


@pytest.mark.parametrize("T", BATCHES)
@pytest.mark.parametrize("E,H,F", [(1, 640, 640), (3, 384, 1152)])
def test_fp32_outputs_keep_every_bit_of_the_hidden_values(T, E, H, F):
    """Hidden values of 23 significant bits in every place of a row, read back one by one."""
    rng = np.random.default_rng(T + F)
    Z = Exact(E, H, F)
    third = (H - 1) // 3
    for e in range(E):
        for f in range(F):   # one of the high, the middle and the low integers each
            Z.up[e, f, 1 + rng.integers(0, third)] = rng.choice([-1, 1])
            Z.up[e, f, 1 + third + rng.integers(0, third)] = rng.choice([-1, 1])
            Z.up[e, f, 1 + 2 * third + rng.integers(0, third)] = rng.choice([-1, 1])
        order = rng.permutation(F)
        Z.down[e, np.arange(H), order[np.arange(H) % F]] = rng.choice([-1, 1], H)
    x = np.zeros((T, H))
    x[:, 1:1 + third] = 65536 * rng.integers(64, 128, (T, third))
    x[:, 1 + third:1 + 2 * third] = 256 * rng.integers(0, 256, (T, third))
    x[:, 1 + 2 * third:1 + 3 * third] = rng.integers(0, 256, (T, third))
    y, want = Z.run(x, torch.bfloat16, "f32", 2.0 ** -3)
    assert np.array_equal(R.f64(y), want)


@pytest.mark.parametrize("T", BATCHES)
@pytest.mark.parametrize("E,H,F", [(1, 640, 640), (3, 384, 1152)])
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
def test_16_bit_outputs_keep_16_bits_of_the_hidden_values(T, E, H, F, xd, yd):
    """Differences of two hidden values of 16 bits whose upper halves are alike."""
    rng = np.random.default_rng(T + F)
    Z = Exact(E, H, F)
    half = (H - 1) // 2
    for e in range(E):
        high = 1 + rng.integers(0, half, F // 2)
        for f in range(F):
            Z.up[e, f, high[f // 2]] = 1
            Z.up[e, f, 1 + half + rng.integers(0, half)] = 1
        pair = rng.permutation(F // 2)[np.arange(H) % (F // 2)]
        sign = rng.choice([-1, 1], H)
        Z.down[e, np.arange(H), 2 * pair] = sign
        Z.down[e, np.arange(H), 2 * pair + 1] = -sign
    x = np.zeros((T, H))
    x[:, 1:1 + half] = 256 * rng.integers(128, 248, (T, half))
    x[:, 1 + half:1 + 2 * half] = rng.integers(0, 256, (T, half))
    y, want = Z.run(x, {"bf16": torch.bfloat16, "f16": torch.float16}[xd], yd, 1.0)
    assert np.abs(want).max() > 0 and np.array_equal(R.f64(y), want)


@pytest.mark.parametrize("T", [1, 3, 5, 20])
@pytest.mark.parametrize("yd", ["f32", "bf16"])
def test_hidden_values_up_to_the_largest_fp32(T, yd):
    """A hidden value between the largest bf16 and the largest fp32 is not an infinity."""
    H, F = 256, 384
    Z = Exact(1, H, F)
    Z.up[0, :, 1] = Z.up[0, :, 2] = 1
    Z.down[0, np.arange(H), np.arange(H)] = np.where(np.arange(H) % 2, 1, -1)
    x = np.zeros((T, H))
    x[:, 1] = 2.0 ** 119 * (2 - 2.0 ** -7)
    x[:, 2] = 2.0 ** 119 * (2.0 ** -7 - 2.0 ** -12)
    y, want = Z.run(x, torch.bfloat16, yd, 2.0 ** -3)
    assert torch.equal(y.cpu(), torch.from_numpy(want).float().to(y.dtype))
