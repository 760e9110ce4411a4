"""Codes of 8-bit activations where the 64-bit quotient is not enough: values that lie next to
a border between two codes by less than it shows, and magnitudes so small that the largest of
them loses bits as an fp32.  The reference decides such values in exact arithmetic."""
from fractions import Fraction

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


def exact_codes(h, w, group):
    """Codes of h w (h [M,K] and w [K] hold fp32 values): 127 h w / a to nearest even, at most 127."""
    p = h * w                                           # 48 bits: exact
    b = R.blocks(p, group)
    a = np.abs(b).max(-1, keepdims=True).astype(np.float32).astype(np.float64)
    v = 127.0 * b / np.where(a > 0, a, 1.0)
    q = np.rint(v)
    near = np.abs(np.abs(v - np.floor(v)) - 0.5) < 2.0 ** -30
    for i in zip(*np.nonzero(near)):
        q[i] = round(127 * Fraction(b[i]) / Fraction(a[i[0], i[1], 0]))   # to nearest, ties to even
    q = np.clip(np.where(a > 0, q, 0.0), -127, 127)
    assert np.abs(q).max() <= 127
    return q.reshape(h.shape).astype(np.int8)


def check(x, w, group, eps=0.0):
    """x [M,K], w [K] fp32 tensors."""
    codes, scales = tern.rms_norm_q8(x.to(DEV), w.to(DEV), eps=eps, group=group)
    want = exact_codes(R.f64(x), R.f64(w), group)
    got = codes.cpu().numpy()
    bad = np.nonzero(got != want)
    assert bad[0].size == 0, (got[bad][:8], want[bad][:8], [i[:8] for i in bad])
    return scales


def near_borders(count, seed):
    """(h, w, A) whose 127 h w / a, a = A 2^24, lies next to a border by so little that its 64-bit
    quotient is the border itself, and rounds to the wrong side."""
    rng = np.random.default_rng(seed)
    found = []
    while len(found) < count:
        n, d = int(rng.integers(70, 127)), int(rng.choice([-1, 1]))
        h = int(rng.integers(1 << 22, 1 << 23)) * 2 + 1
        m = (2 * n + 1) << 23
        if h % 127 == 0 or np.gcd(127 * h, m) > 1:
            continue
        w = d * pow(127 * h, -1, m) % m                 # 127 h w = d + A m
        A = (127 * h * w - d) // m
        if w >= 1 << 24 or not 1 << 20 <= A < 1 << 24:
            continue
        if np.rint(127.0 * (float(h) * float(w)) / (A * 2.0 ** 24)) != round(Fraction(127 * h * w, A << 24)):
            found.append((h, w, A))
    return found


@pytest.mark.parametrize("K,group", [(K, g) for K in (5, 8, 100, 128, 384, 1000, 5119, 12288, 20000, 40000) for g in (0, 128) if g == 0 or K % g == 0])
def test_borders_that_64_bits_do_not_show(K, group):
    print(f"borders K={K} group={group}", flush=True)
    cases = [(11742707, 12087109, 14819600)] + near_borders(12, 7)
    for h, w, A in cases:
        x, ww = torch.zeros((2, K)), torch.full((K,), 1.0)
        for s in ([0] if not group else range(0, K, 128)):   # every block's
            x[0, s], ww[s] = A, 2.0 ** 24
            x[0, s + 3], ww[s + 3] = h, w
            x[1, s], x[1, s + 3] = -A, -h
        check(x, ww, group)


@pytest.mark.parametrize("K,group", [(K, g) for K in (4, 17, 128, 512, 1280, 9000, 20000, 40000) for g in (0, 128) if g == 0 or K % g == 0])
def test_codes_of_magnitudes_below_the_normal_range(K, group):
    """The largest magnitude as an fp32 is up to a third below the value: its code is 127, not 178."""
    print(f"small magnitudes K={K} group={group}", flush=True)
    rng = np.random.default_rng(K)
    for top in (1.4, -1.4, 1.49, 2.4, 3.49, -7.4, 12.5, 100.3):
        x = torch.from_numpy(rng.uniform(-1, 1, (3, K))).float() * 2.0 ** -100
        w = torch.full((K,), abs(top) * 2.0 ** -49)
        x[:, ::3] = 2.0 ** -100 if top > 0 else -2.0 ** -100
        check(x, w, group)


def test_codes_of_quantize_below_the_normal_range():
    x = torch.from_numpy(np.random.default_rng(1).integers(-9, 10, (4, 256)) * 2.0 ** -149).float()
    for group in (0, 128):
        codes, _ = tern.q8_quantize(x.to(DEV), group=group)
        assert np.array_equal(codes.cpu().numpy(), exact_codes(R.f64(x), np.ones(256), group))


@pytest.mark.parametrize("M,K", [(50, 128), (9, 1000), (7, 5120), (3, 20000), (2, 40000)])
def test_codes_of_ordinary_values(M, K):
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K))).float()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(K)).float()
    for group in ((0,) if K % 128 else (0, 128)):
        check(x, w, group, 1e-6)
