"""The product of 8-bit activations with ternary weights on the GPU: against a 64-bit
reference, bit for bit where the arithmetic is exact, and next to the norm that
feeds it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import q8_util as R  # noqa: E402

tern = pytest.importorskip("ternary_weight_matmul_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def problem(M, N, K, group, seed, lo=-127):
    rng = np.random.default_rng(seed)
    q = rng.integers(lo, 128, (M, K)).astype(np.int8)
    xs = np.exp(rng.uniform(-6, 0, (M, K // 128 if group else 1))).astype(np.float32)
    packed = rng.integers(0, 256, (N, K // 4)).astype(np.uint8)   # with the reserved code 11
    ws = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), (N, K // 128))).astype(np.float16)
    return q, xs, packed, ws


def run(q, xs, packed, ws, yd):
    M, N = q.shape[0], packed.shape[0]
    buf = torch.full((M * N + 64,), float("nan"), dtype=DT[yd], device=DEV)
    y = buf[:M * N].view(M, N)
    tern.matmul_q8_into(dev(q), dev(xs), dev(packed), dev(ws), y)
    torch.cuda.synchronize()
    assert torch.isnan(buf[M * N:]).all()
    return y


# rows on either side of every tile and choice; odd columns; one block of K to many
SIZES = [(1, 1, 128), (1, 16, 128), (1, 5, 640), (1, 513, 1152), (1, 5120, 512), (2, 33, 384), (2, 1000, 5120), (3, 100, 1408),
         (3, 4099, 256), (4, 17, 17408), (4, 260, 2048), (4, 20000, 128), (5, 64, 896), (5, 1001, 640), (7, 31, 2176),
         (8, 129, 4096), (9, 48, 1280), (12, 515, 640), (15, 64, 17408), (16, 1000, 1152), (16, 17, 128), (16, 17000, 256),
         (17, 65, 384), (24, 511, 640), (31, 129, 1024), (32, 700, 896), (33, 257, 256), (37, 1001, 1152), (48, 64, 5120),
         (63, 200, 128), (64, 640, 640), (65, 96, 768), (100, 1111, 2080 // 128 * 128), (127, 129, 384),
         (128, 1280, 1280), (129, 513, 512), (200, 4100, 256), (257, 300, 2688), (300, 768, 1152), (513, 1030, 384)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group,yd", [(0, "bf16"), (128, "f32"), (0, "f16"), (128, "bf16")])
def test_product(M, N, K, group, yd):
    print(f"matmul_q8 M={M} N={N} K={K} group={group} -> {yd}", flush=True)
    p = problem(M, N, K, group, M + N + K)
    want, bound = R.product(*p, DT[yd])
    R.assert_close(run(*p, yd), want, bound, "matmul_q8")


@pytest.mark.parametrize("M", [1, 2, 3, 4, 6, 11, 16, 20, 40, 70, 130, 300])
@pytest.mark.parametrize("group", [0, 128])
def test_exact_arithmetic(M, group):
    """Power-of-two scales: every step is exact, the largest sums and the code -128 among them."""
    K, N = 1024, 300
    rng = np.random.default_rng(M)
    q, xs, packed, ws = problem(M, N, K, group, M, lo=-128)
    q[0] = -128
    packed[:3] = [[0x55], [0xAA], [0xFF]]   # all +1, all -1, all of the reserved code
    xs = np.exp2(rng.integers(-2, 3, xs.shape)).astype(np.float32)
    ws = np.exp2(rng.integers(-3, 2, ws.shape)).astype(np.float16)
    want, _ = R.product(q, xs, packed, ws, torch.float32)
    got = R.f64(run(q, xs, packed, ws, "f32"))
    assert np.array_equal(got, want)
    assert (got[:, 2] == 0).all()


@pytest.mark.parametrize("M,N,K", [(1, 40, 640), (4, 40, 512), (9, 70, 384), (16, 40, 640), (30, 64, 256), (70, 150, 640),
                                   (260, 270, 384)])
def test_every_place_of_a_weight(M, N, K):
    """One weight a row, at every k in turn: an activation is met by its own weight only."""
    q, xs, packed, ws = problem(M, N, K, 0, 1)
    xs[:] = 1
    ws[:] = 1
    for k0 in range(0, K, N):
        t = np.zeros((N, K), dtype=np.int64)
        for n in range(N):
            if k0 + n < K:
                t[n, k0 + n] = 1 if n % 2 == 0 else -1
        got = R.f64(run(q, xs, R.pack_ternary(t), ws, "f32"))
        assert np.array_equal(got, q.astype(np.float64) @ t.T)


@pytest.mark.parametrize("M", [1, 4, 10, 16, 33, 150])
def test_infinities_and_nans_stay_in_their_row_and_column(M):
    N, K = 200, 640
    for group in (0, 128):
        q, xs, packed, ws = problem(M, N, K, group, M + group)
        clean, bound = R.product(q, xs, packed, ws, torch.float32)
        xs[M // 2, -1] = np.nan
        ws[17, 2] = np.inf
        ws[50, 4] = np.nan
        y = R.f64(run(q, xs, packed, ws, "f32"))
        rows, cols = np.arange(M) != M // 2, ~np.isin(np.arange(N), (17, 50))
        assert np.isnan(y[M // 2]).all() and np.isnan(y[:, 50]).all() and not np.isfinite(y[:, 17]).any()
        assert (np.abs(y - clean) <= bound)[np.ix_(rows, cols)].all()


def test_zero_scales_and_codes():
    q, xs, packed, ws = problem(6, 64, 512, 128, 3)
    q[2] = 0
    xs[3] = 0
    ws[5] = 0
    y = run(q, xs, packed, ws, "bf16")
    assert (y[2] == 0).all() and (y[3] == 0).all() and (y[:, 5] == 0).all()


def test_sizes_of_zero():
    for M, N, K in ((0, 5, 128), (3, 0, 128), (3, 5, 0)):
        y = tern.matmul_q8(dev(np.zeros((M, K), np.int8)), dev(np.ones((M, 1), np.float32)),
                           dev(np.zeros((N, K // 4), np.uint8)), dev(np.zeros((N, K // 128), np.float16)))
        assert y.shape == (M, N) and (y == 0).all()


@pytest.mark.parametrize("M,N", [(1, 31), (4, 33), (16, 31), (40, 35), (200, 33)])
def test_scales_and_outputs_at_any_address(M, N):
    K = 384
    q, xs, packed, ws = problem(M, N, K, 128, M)
    s = torch.zeros(ws.size + 1, dtype=torch.float16, device=DEV)
    s[1:] = dev(ws).view(-1)
    y = torch.full((M * N + 2,), float("nan"), dtype=torch.bfloat16, device=DEV)
    tern.matmul_q8_into(dev(q), dev(xs), dev(packed), s[1:].view(N, K // 128), y[1:1 + M * N].view(M, N))
    want, bound = R.product(q, xs, packed, ws, torch.bfloat16)
    R.assert_close(y[1:1 + M * N].view(M, N), want, bound)
    assert torch.isnan(y[0]) and torch.isnan(y[-1])


@pytest.mark.parametrize("M", [1, 3, 16, 50, 140])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_to_product(M, group):
    """A norm's 8-bit outputs through the product, as they are used; the two together agree with
    the product in 16 bits to what 8 bits lose."""
    K, N = 5120, 640
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16)
    r = torch.from_numpy(rng.standard_normal((M, K)) * 3).to(torch.bfloat16)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(K)).float()
    _, _, packed, ws = problem(1, N, K, 0, M)
    codes, scales, h = tern.rms_norm_q8(x.to(DEV), w.to(DEV), residual=r.to(DEV), group=group)
    y = tern.matmul_q8(codes, scales, dev(packed), dev(ws), out_dtype=torch.float32)
    _, _, v, f = R.norm(x, w, 1e-6, r)
    q, _ = R.quantize(v, f, group)
    want, bound = R.product(q, R.f64(scales), packed, ws, torch.float32)
    R.assert_close(y, want, bound, "norm to product")
    normed = v * f[:, None]
    half = np.repeat(R.f64(scales), K // scales.shape[1], axis=1) * 0.5001   # half a step of 8 bits
    exact = normed @ R.dense(packed, ws).T
    assert (np.abs(R.f64(y) - exact) <= half @ np.abs(R.dense(packed, ws)).T + bound).all()


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_a_graph_and_another_stream(M):
    q, xs, packed, ws = problem(M, 1000, 1280, 0, M)
    d = [dev(a) for a in (q, xs, packed, ws)]
    want = tern.matmul_q8(*d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = tern.matmul_q8(*d)
    side.synchronize()
    assert torch.equal(y, want)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = tern.matmul_q8(*d)
    with torch.cuda.graph(g2):
        y2 = tern.matmul_q8(*d, out_dtype=torch.float32)
    for seed in (5, 6, 7):
        d[0].copy_(dev(problem(M, 1000, 1280, 0, seed)[0]))
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tern.matmul_q8(*d)) and torch.equal(y2, tern.matmul_q8(*d, out_dtype=torch.float32))


# Large products have a kernel of their own, with a workspace.
LARGE = (1100, 7501, 2816)


@pytest.mark.parametrize("group,yd,odd", [(0, "bf16", 1), (128, "f32", 1), (128, "f16", 0), (0, "f32", 0)])
@pytest.mark.parametrize("more", [0, 128])   # an even and an odd number of blocks: codes come for two at a time
def test_large_product(group, yd, odd, more):
    M, N, K = LARGE
    N -= 1 - odd
    K += more
    assert tern.lib.tern_matmul_q8_workspace(M, N, K) > 0
    print(f"matmul_q8 M={M} N={N} K={K} group={group} -> {yd}", flush=True)
    q, xs, packed, ws = problem(M, N, K, group, M + group, lo=-128)
    want, bound = R.product(q, xs, packed, ws, DT[yd])
    R.assert_close(run(q, xs, packed, ws, yd), want, bound, "matmul_q8")


def test_large_product_exact_and_every_place_of_a_weight():
    """Power-of-two scales and one weight a row, at every k."""
    M, N, K = LARGE
    rng = np.random.default_rng(1)
    q = rng.integers(-128, 128, (M, K)).astype(np.int8)
    q[3] = -128
    t = np.zeros((N, K), dtype=np.int64)
    t[np.arange(N), np.arange(N) % K] = np.where(np.arange(N) % 3 == 0, -1, 1)
    t[-2], t[-1] = 1, -1
    xs = np.exp2(rng.integers(-2, 3, (M, K // 128))).astype(np.float32)
    ws = np.exp2(rng.integers(-3, 2, (N, K // 128))).astype(np.float16)
    packed = R.pack_ternary(t)
    want, _ = R.product(q, xs, packed, ws, torch.float32)
    assert np.array_equal(R.f64(run(q, xs, packed, ws, "f32")), want)


def test_large_product_infinities_and_nans_stay_in_their_row_and_column():
    M, N, K = LARGE
    q, xs, packed, ws = problem(M, N, K, 128, 9)
    clean = R.f64(run(q, xs, packed, ws, "f32"))
    xs[M // 2, -1] = np.nan
    ws[17, 2] = np.inf
    ws[N - 1, 4] = np.nan
    y = R.f64(run(q, xs, packed, ws, "f32"))
    rows, cols = np.arange(M) != M // 2, ~np.isin(np.arange(N), (17, N - 1))
    assert np.isnan(y[M // 2]).all() and np.isnan(y[:, N - 1]).all() and not np.isfinite(y[:, 17]).any()
    assert np.array_equal(y[np.ix_(rows, cols)], clean[np.ix_(rows, cols)])


def test_large_products_in_two_graphs_and_on_two_streams():
    M, N, K = LARGE
    p = [[dev(a) for a in problem(M, N, K, 0, seed)] for seed in (1, 2)]
    want = [tern.matmul_q8(*d) for d in p]
    sides = [torch.cuda.Stream() for _ in p]
    torch.cuda.synchronize()
    got = []
    for d, side in zip(p, sides):
        with torch.cuda.stream(side):
            got.append([tern.matmul_q8(*d) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)
    graphs = [torch.cuda.CUDAGraph() for _ in p]
    out = []
    for d, g in zip(p, graphs):
        with torch.cuda.graph(g):
            out.append(tern.matmul_q8(*d))
    for _ in range(3):
        for y in out:
            y.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(out, want))


# which of the kernels for more than 4 rows takes a size: few rows, 64 x 128 and 128 x 384 tiles, the
# first two on either side of what the first can take (K >= 512)
@pytest.mark.parametrize("M,N,K", [(5, 700, 384), (32, 1000, 384), (33, 640, 512), (65, 3000, 512), (97, 5120, 640),
                                   (600, 1000, 384), (900, 2000, 640), (520, 5121, 1152)])
@pytest.mark.parametrize("group", [0, 128])
def test_rows_do_not_touch_each_other(M, N, K, group):
    """Every row alone gives what it gives in the batch, to the last bits' order of sums; rows behind
    the last stay as they were, and twice the same call is the same to the bit."""
    print(f"matmul_q8 M={M} N={N} K={K} group={group}", flush=True)
    q, xs, packed, ws = problem(M, N, K, group, M)
    d = [dev(a) for a in (q, xs, packed, ws)]
    y = run(q, xs, packed, ws, "f32")
    assert torch.equal(y, tern.matmul_q8(*d, out_dtype=torch.float32))
    rows = [0, M // 2, M - 1]
    want, bound = R.product(q[rows], xs[rows], packed, ws, torch.float32)
    R.assert_close(y[rows], want, bound, "rows of the batch")
    R.assert_close(tern.matmul_q8(d[0][rows], d[1][rows], *d[2:], out_dtype=torch.float32), want, bound, "rows alone")
