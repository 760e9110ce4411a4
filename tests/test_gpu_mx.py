"""Microscaled 4-bit floats on the GPU: quantisation bit for bit, the products
against 64-bit references and, where the arithmetic is exact, bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mx_util as R  # noqa: E402

tern = pytest.importorskip("ternary_weight_matmul_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def same_bits(t, a):
    return np.array_equal(t.cpu().numpy(), a)


# --- quantisation ---------------------------------------------------------------

@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (1, 5120), (65, 1056), (2, 32 * 257), (1025, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_quantize_bits(M, K, dt):
    print(f"quantize {M}x{K} {dt}", flush=True)
    rng = np.random.default_rng(M * K)
    x = torch.from_numpy(rng.standard_normal((M, K)) * np.exp2(rng.integers(-12, 12, (M, 1)))).to(DT[dt])
    codes, exps = tern.mx_quantize(x.to(DEV))
    c, e = R.quantize(R.f64(x))
    assert same_bits(exps, e)
    assert same_bits(codes, R.pack_nibbles(c))
    for od in DT:
        got = tern.mx_dequant(codes, exps, out_dtype=DT[od])
        want = torch.from_numpy(R.values(R.pack_nibbles(c), e)).float().to(DT[od])
        assert torch.equal(got.cpu(), want)


def test_quantize_borders():
    """Every border between two codes, one step below and above, of either sign, at small,
    ordinary and extreme scales; ties go to the even code."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.999])
    rows = []
    for E in (-126, -100, -3, 0, 5, 120):
        b = (borders * 2.0 ** E).astype(np.float32)
        v = np.concatenate([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(np.inf))])
        v = np.concatenate([v, -v])
        for i in range(0, v.size, 28):
            row = np.zeros(32, dtype=np.float32)
            part = v[i:i + 28]
            row[:part.size] = part
            row[28] = 4.0 * 2.0 ** E   # pins the scale to 2^E
            rows.append(np.where(np.abs(row) >= 8.0 * 2.0 ** E, 0, row))
    x = np.stack(rows)
    codes, exps = tern.mx_quantize(dev(x))
    c, e = R.quantize(x.astype(np.float64))
    assert same_bits(exps, e) and same_bits(codes, R.pack_nibbles(c))


def test_quantize_extremes():
    """Zeros, subnormals, the largest values, infinities and NaN: a block with one of the last
    two reads back as NaN, its neighbours stay."""
    x = np.zeros((8, 64), dtype=np.float32)
    x[1, 0] = 2.0 ** -149
    x[2, :] = 2.0 ** -127
    x[3, 5] = np.finfo(np.float32).max
    x[4, 3] = np.inf
    x[5, 40] = -np.inf
    x[6, 7] = np.nan
    x[7, :] = -0.0
    x[4:7, 32:40] += 1.5
    codes, exps = tern.mx_quantize(dev(x))
    c, e = R.quantize(x.astype(np.float64))
    assert same_bits(exps, e) and same_bits(codes, R.pack_nibbles(c))
    v = R.f64(tern.mx_dequant(codes, exps))
    assert np.isnan(v[4, :32]).all() and np.isfinite(v[4, 32:]).all()
    assert np.isnan(v[5, 32:]).all() and np.isfinite(v[5, :32]).all()
    assert np.isnan(v[6, :32]).all()
    assert not np.isnan(v[[0, 1, 2, 3, 7]]).any()


def test_dequant_every_code_and_exponent():
    codes = np.tile(np.arange(256, dtype=np.uint8)[None, :], (256, 1))   # 512 values = 16 blocks
    exps = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 16))
    for od, dt in DT.items():
        got = tern.mx_dequant(dev(codes), dev(exps), out_dtype=dt).cpu()
        with np.errstate(over="ignore"):
            want = torch.from_numpy(R.values(codes, exps).astype(np.float32)).to(dt)
        assert torch.equal(torch.isnan(got), torch.isnan(want)), od
        keep = ~torch.isnan(want)
        assert torch.equal(got[keep], want[keep]), od


# --- products -------------------------------------------------------------------

def weights(N, K, seed, spread=6):
    """Random codes and exponents: every code, scales over `spread` binades."""
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (N, K // 2)).astype(np.uint8),
            (120 + rng.integers(0, spread, (N, K // 32))).astype(np.uint8))


def activations(M, K, dt, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K))
    x[rng.random((M, K)) < 0.01] *= 20
    return torch.from_numpy(x).to(DT[dt])


def nan_out(M, N, yd):
    return torch.full((M, N), float("nan"), dtype=DT[yd], device=DEV)


# every M from 1 to 17 somewhere, one block to many steps, N of one row, off the tiles
@pytest.mark.parametrize("M,K,yd", [(4200, 4096, "bf16"), (4201, 4160, "f32"), (5000, 4128, "f16")])
def test_dequant_past_the_caches(M, K, yd):
    print(f"mx_dequant {M}x{K} -> {yd}", flush=True)
    codes, exps = weights(M, K, M + K, spread=6)
    y = tern.mx_dequant(dev(codes), dev(exps), DT[yd])
    assert torch.equal(y.cpu(), torch.from_numpy(np.asarray(R.values(codes, exps))).to(DT[yd]))


SHAPES = [(1, 1, 32), (1, 5120, 5120), (2, 17, 64), (3, 33, 96), (4, 1000, 1056), (5, 16, 256), (6, 31, 288),
          (7, 300, 4128), (8, 129, 8192), (9, 100, 512), (10, 8, 544), (11, 95, 17408), (12, 7, 640), (13, 130, 32),
          (14, 257, 1024), (15, 64, 2080), (16, 500, 5120), (17, 48, 320), (31, 77, 1184), (33, 40, 768),
          (64, 257, 1056), (65, 300, 2048), (100, 515, 352), (127, 128, 4096), (128, 256, 512), (129, 513, 544),
          (200, 700, 1312), (257, 1030, 2080), (300, 260, 160), (512, 1024, 1024),
          (32, 6000, 128), (160, 1111, 96), (161, 300, 2080), (700, 9300, 96), (641, 9411, 544), (1030, 6100, 1056)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_matmul(M, N, K, xd, yd):
    print(f"mx_matmul {M}x{K}->{N} {xd}->{yd}", flush=True)
    codes, exps = weights(N, K, M + N + K)
    x = activations(M, K, xd, M * 7 + K)
    y = tern.mx_matmul_into(x.to(DEV), dev(codes), dev(exps), nan_out(M, N, yd))
    X, W = R.f64(x), R.values(codes, exps)
    want = X @ W.T
    R.assert_close(y, want, R.product_bound(X, W, want, DT[yd]), "mx_matmul")


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("yd", ["bf16", "f32", "f16"])
def test_matmul_mx(M, N, K, yd):
    print(f"mx_matmul_mx {M}x{K}->{N} ->{yd}", flush=True)
    codes, exps = weights(N, K, M + N + K)
    xc, xe = weights(M, K, M * 3 + N, spread=4)
    y = tern.mx_matmul_mx_into(dev(xc), dev(xe), dev(codes), dev(exps), nan_out(M, N, yd))
    X, W = R.values(xc, xe), R.values(codes, exps)
    want = X @ W.T
    R.assert_close(y, want, R.product_bound(X, W, want, DT[yd]), "mx_matmul_mx")


@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_largest_k(kind):
    """Offsets of a row near 2^24 values, with sums that are exact: ones and halves, few of them."""
    M, N, K = 2, 73, 1 << 24
    print(f"K = 2^24 {kind}", flush=True)
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    exps = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    at = torch.arange(0, K // 2, 4099, device=DEV)
    codes[:, at] = 0x12          # 1 and 0.5
    codes[:, -1] = 0x21
    codes[72, -1] = 0
    x = torch.ones((M, K), dtype=torch.bfloat16, device=DEV)
    x[1] = 2
    if kind == "mx":
        y = tern.mx_matmul_mx(*tern.mx_quantize(x), codes, exps, torch.float32)
    else:
        y = tern.mx_matmul(x, codes, exps, torch.float32)
    n = at.numel() + (0 if int(at[-1]) == K // 2 - 1 else 1)
    want = torch.full((M, N), 1.5 * n)
    want[:, 72] -= 1.5
    want[1] *= 2
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f16", "mx"])
def test_exact_arithmetic(M, N, K, kind):
    """Small integer activations and one scale per row: every partial sum is a multiple of
    half the scale and exact in fp32 in any order, so the outputs are too."""
    rng = np.random.default_rng(M + 5 * N + K)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    exps = np.repeat((110 + rng.integers(0, 30, (N, 1))).astype(np.uint8), K // 32, axis=1)
    if kind == "mx":
        xc = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
        xe = np.full((M, K // 32), 127, dtype=np.uint8)
        X = R.values(xc, xe)
        y = tern.mx_matmul_mx_into(dev(xc), dev(xe), dev(codes), dev(exps), nan_out(M, N, "f32"))
    else:
        X = rng.integers(-16, 17, (M, K)).astype(np.float64)
        y = tern.mx_matmul_into(torch.from_numpy(X).to(DT[kind]).to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    assert np.array_equal(R.f64(y), X @ R.values(codes, exps).T)


@pytest.mark.parametrize("M,N,K", [(1, 40, 1056), (8, 40, 512), (16, 70, 96), (40, 130, 288), (300, 600, 544)])
@pytest.mark.parametrize("xd", ["f16", "bf16"])
def test_every_block_has_its_own_scale(M, N, K, xd):
    """One-hot activations read single weights back, through scales over the whole fp32 range."""
    rng = np.random.default_rng(K)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    exps = rng.integers(8, 240, (N, K // 32)).astype(np.uint8)
    X = np.zeros((M, K))
    X[np.arange(M), rng.integers(0, K, M)] = rng.choice([1.0, -2.0, 0.5], M)
    y = tern.mx_matmul_into(torch.from_numpy(X).to(DT[xd]).to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    want = (X @ R.values(codes, exps).T).astype(np.float32)
    # fp32 subnormal results may be flushed by the matrix cores
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("M,N,K", [(1, 24, 512), (4, 24, 512), (8, 24, 512), (20, 40, 256), (300, 300, 256)])
@pytest.mark.parametrize("xd", ["f16", "bf16"])
def test_fp16_activations_keep_every_bit(M, N, K, xd):
    """Activations with a full significand and large and small magnitudes side by side."""
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.uniform(1, 2, (M, K)) * np.exp2(rng.integers(-13, 14, (M, K)))).to(DT[xd])
    codes, exps = weights(N, K, M, spread=1)
    y = tern.mx_matmul_into(x.to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    X, W = R.f64(x), R.values(codes, exps)
    want = X @ W.T
    R.assert_close(y, want, R.product_bound(X, W, want, torch.float32))


@pytest.mark.parametrize("M,N,K", [(3, 40, 288), (16, 40, 288), (70, 300, 288), (300, 600, 544)])
@pytest.mark.parametrize("xd", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_values_stay_in_their_row_and_column(M, N, K, xd, bad):
    codes, exps = weights(N, K, 5)
    x = activations(M, K, xd, 6)
    clean = tern.mx_matmul(x.to(DEV), dev(codes), dev(exps), out_dtype=torch.float32)
    x[M - 1, K - 1] = bad
    exps[N - 1, 0] = 255
    y = tern.mx_matmul_into(x.to(DEV), dev(codes), dev(exps), nan_out(M, N, "f32"))
    assert torch.equal(y[:M - 1, :N - 1], clean[:M - 1, :N - 1])
    assert not torch.isfinite(y[M - 1]).any()
    assert torch.isnan(y[:, N - 1]).all()


@pytest.mark.parametrize("M,N,K", [(3, 40, 288), (16, 40, 288), (300, 600, 544)])
def test_nan_blocks_of_4_bit_activations(M, N, K):
    codes, exps = weights(N, K, 5)
    xc, xe = weights(M, K, 6)
    clean = tern.mx_matmul_mx(dev(xc), dev(xe), dev(codes), dev(exps), out_dtype=torch.float32)
    xe[M - 1, K // 32 - 1] = 255
    y = tern.mx_matmul_mx_into(dev(xc), dev(xe), dev(codes), dev(exps), nan_out(M, N, "f32"))
    assert torch.equal(y[:M - 1], clean[:M - 1])
    assert torch.isnan(y[M - 1]).all()


@pytest.mark.parametrize("M", [1, 8, 24, 300])
def test_output_neighbours_are_untouched(M):
    """Writes stay inside Y: the elements before and behind it keep their values."""
    N, K = 333, 160
    codes, exps = weights(N, K, 1)
    x = activations(M, K, "bf16", 2).to(DEV)
    buf = torch.full((64 + M * N + 4096,), 7.0, dtype=torch.float32, device=DEV)
    y = buf[64:64 + M * N].view(M, N)
    tern.mx_matmul_into(x, dev(codes), dev(exps), y)
    assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()
    assert torch.equal(y, tern.mx_matmul(x, dev(codes), dev(exps), out_dtype=torch.float32))


def test_misaligned_and_strided_inputs_are_refused():
    codes, exps = (dev(a) for a in weights(16, 64, 1))
    x = activations(4, 72, "bf16", 2).to(DEV)
    with pytest.raises(ValueError):
        tern.mx_matmul(x[:, :64], codes, exps)
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 64)
    with pytest.raises(tern.TernError):
        tern.mx_matmul(flat, codes, exps)
    with pytest.raises(tern.TernError):
        tern.mx_quantize(flat)
    with pytest.raises(ValueError):
        tern.mx_quantize(x.t())
    with pytest.raises(tern.TernError):
        tern.mx_quantize(x[:, :40].contiguous())
    with pytest.raises(ValueError):
        tern.mx_matmul(x, codes, exps)
    with pytest.raises(ValueError):
        tern.mx_matmul(x[:, :64].contiguous(), codes, exps.cpu())


@pytest.mark.parametrize("M,N,K", [(1, 130, 1024), (7, 33, 1056), (40, 700, 2048), (200, 301, 352), (641, 9411, 96)])
@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_scales_and_outputs_at_any_address(M, N, K, kind):
    """Exponent bytes at an odd address and outputs at an odd element give the same bits."""
    print(f"addresses {M}x{K}->{N} {kind}", flush=True)
    codes, exps = (dev(t) for t in weights(N, K, M + K))
    xc, xe = (dev(t) for t in weights(M, K, M + N, spread=4))
    x = activations(M, K, "bf16", M).to(DEV)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        flat.copy_(t.reshape(-1))
        return flat.view(t.shape)

    def product(ex, xex, out):
        return (tern.mx_matmul_into(x, codes, ex, out) if kind == "bf16"
                else tern.mx_matmul_mx_into(xc, xex, codes, ex, out))

    for yd in (torch.bfloat16, torch.float32):
        want = product(exps, xe, torch.empty((M, N), dtype=yd, device=DEV))
        got = product(shifted(exps), shifted(xe), shifted(torch.zeros((M, N), dtype=yd, device=DEV)))
        assert torch.equal(got, want)
    assert torch.equal(tern.mx_dequant(codes, shifted(exps)), tern.mx_dequant(codes, exps))


def test_empty_sizes():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    c, s = tern.mx_quantize(e)
    assert c.shape == (0, 32) and s.shape == (0, 2)
    codes, exps = (dev(a) for a in weights(16, 64, 1))
    assert tern.mx_matmul(e, codes, exps).shape == (0, 16)
    z = tern.mx_matmul(torch.empty((3, 0), dtype=torch.bfloat16, device=DEV),
                       torch.empty((5, 0), dtype=torch.uint8, device=DEV),
                       torch.empty((5, 0), dtype=torch.uint8, device=DEV))
    assert z.shape == (3, 5) and (z == 0).all()


@pytest.mark.parametrize("M", [1, 12, 300])
def test_another_stream_and_graph_replays(M):
    """Calls follow the current stream; a captured quantise-and-multiply replays on new inputs,
    with eager work between the replays."""
    N, K = 640, 1056
    codes, exps = (dev(a) for a in weights(N, K, 3))
    xs = [activations(M, K, "bf16", s).to(DEV) for s in range(4)]
    want = [(tern.mx_matmul(x, codes, exps), tern.mx_matmul_mx(*tern.mx_quantize(x), codes, exps)) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tern.mx_matmul(xs[0], codes, exps)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0][0])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = tern.mx_matmul(x, codes, exps)
        b = tern.mx_matmul_mx(*tern.mx_quantize(x), codes, exps)
    for i in (1, 2, 3, 1):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])
        assert torch.equal(tern.mx_matmul(xs[i], codes, exps), want[i][0])


def test_long_rows_and_many_rows_pass_32_bits():
    """More than 2^32 bytes of weights: the last rows are read at their own place."""
    N, K = 17000, 524288
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    exps = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    codes[N - 1, K // 2 - 1] = 0x70    # the last element is 6
    codes[N - 2, 0] = 0x03             # the first one is 1.5
    for M in (1, 300):
        x = torch.ones((M, K), dtype=torch.bfloat16, device=DEV)
        y = tern.mx_matmul(x, codes, exps, out_dtype=torch.float32)
        assert (y[:, N - 1] == 6).all() and (y[:, N - 2] == 1.5).all() and (y[:, :N - 2] == 0).all()
