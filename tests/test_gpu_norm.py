"""The root-mean-square norm with its residual addition and 8-bit outputs, and the
conversion of 8-bit activations, on the GPU: against a 64-bit reference, bit for
bit where a result is exact."""
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


def values(shape, dtype, seed, big=0.02):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape)
    v = np.where(rng.random(shape) < big, v * 8, v)
    return torch.from_numpy(v).to(DT[dtype])


def equal_scales(got, want):
    """Formed in 64 bits, rounded once: off by half a step, and by a bit of the 64-bit sum's order."""
    g = R.f64(got)
    assert g.shape == want.shape
    same = (np.isnan(g) & np.isnan(want)) | (np.abs(g - want) <= np.abs(want) * R.STEP * 1.001 + 2.0 ** -149)
    assert same.all(), (g[~same][:4], want[~same][:4])


def run(x, w, eps, r, group, yd, coded=True):
    """The general form into guarded buffers; (y, codes, scales, h) on the CPU."""
    M, K = x.shape
    xd = x.to(DEV)
    rd = r.to(DEV) if r is not None else None
    wd = w.to(DEV) if w is not None else None
    guard = 64
    yb = torch.full((M * K + guard,), 7.0, dtype=DT[yd], device=DEV)
    cb = torch.full((M * K + guard,), 77, dtype=torch.int8, device=DEV)
    G = K // group if group else 1
    sb = torch.full((M * G + guard,), 7.0, device=DEV)
    hb = torch.full((M * K + guard,), 7.0, dtype=r.dtype, device=DEV) if r is not None else None
    y, c, s = yb[:M * K].view(M, K), cb[:M * K].view(M, K), sb[:M * G].view(M, G)
    h = hb[:M * K].view(M, K) if hb is not None else None
    tern.rms_norm_into(xd, wd, out=y, codes=c if coded else None, scales=s if coded else None, eps=eps, residual=rd,
                       residual_out=h)
    torch.cuda.synchronize()
    assert (yb[M * K:] == 7).all() and (cb[M * K:] == 77).all() and (sb[M * G:] == 7).all()
    assert hb is None or (hb[M * K:] == 7).all()
    return y.cpu(), c.cpu(), s.cpu(), h.cpu() if h is not None else None


def check(x, w, eps, r, group, yd):
    y, c, s, h = run(x, w, eps, r, group, yd)
    wh, wy, v, f = R.norm(x, w, eps, r)
    if h is not None:
        assert np.array_equal(R.f64(h), wh)
    R.assert_close(y, wy, R.norm_bound(wy, DT[yd]), "norm")
    q, ws = R.quantize(v, f, group)
    assert np.array_equal(c.numpy(), q)
    equal_scales(s, ws)


# rows of every way in which they are held: 16 lanes, a wave, 256 to 1024 threads, on and off the borders
SIZES = [(1, 1), (2, 3), (3, 7), (5, 8), (70, 15), (33, 100), (17, 128), (9, 129), (5, 512), (3, 513), (7, 1000),
         (2, 1024), (3, 1025), (2, 2048), (3, 2049), (4, 4095), (2, 4097), (3, 5120), (2, 6145), (1, 8195), (2, 12288),
         (1, 12289), (2, 17408), (1, 20481), (2, 32768), (1, 32769), (1, 65536), (9001, 40), (40000, 17), (2500, 640)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("xd,rd,wd,yd", [("bf16", "bf16", "bf16", "bf16"), ("f16", "f32", "f32", "f32"),
                                         ("bf16", None, "f32", "f32"), ("f32", "f32", None, "bf16"),
                                         ("f16", "f16", "f16", "f16"), ("f32", None, "bf16", "f16"),
                                         ("bf16", "f32", "f32", "bf16"), ("f16", None, None, "f16")])
def test_norm(M, K, xd, rd, wd, yd):
    print(f"norm M={M} K={K} x {xd} residual {rd} weight {wd} -> {yd}", flush=True)
    x = values((M, K), xd, M + K)
    r = (values((M, K), rd, M + K + 1) * 4).to(DT[rd]) if rd else None
    w = (values((1, K), "f32", K, 0)[0] * 0.3 + 1).to(DT[wd]) if wd else None
    check(x, w, 1e-6, r, 0, yd)


@pytest.mark.parametrize("M,K", [(1, 128), (50, 128), (3, 256), (2, 640), (5, 1024), (3, 2048), (2, 5120), (3, 8192),
                                 (2, 17408), (1, 32768), (1, 65536), (3000, 384)])
@pytest.mark.parametrize("xd,rd", [("bf16", "bf16"), ("f16", None), ("f32", "f32")])
def test_a_scale_per_128(M, K, xd, rd):
    print(f"norm M={M} K={K} {xd} {rd} group 128", flush=True)
    x = values((M, K), xd, M + K)
    r = values((M, K), rd, M + K + 1) if rd else None
    w = (values((1, K), "f32", K, 0)[0] * 0.3 + 1).to(DT["f32" if rd else xd])
    check(x, w, 1e-5, r, 128, "bf16")


@pytest.mark.parametrize("xd", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("group", [0, 128])
def test_codes_on_their_borders(xd, group):
    """Values that lie exactly between two codes, for largest magnitudes whose reciprocal is not exact."""
    K = 512
    rows = []
    for top in (254, 127, 253, 3, 191, 85, 251):
        v = np.arange(K) % (2 * top + 1) - top
        rows.append(np.where(np.arange(K) % 128 == 5, top, v))
        # 127 v / top = n + 1/2 exactly: v = top (2 n + 1) / 254
        n = np.arange(K) % 253 - 127
        t = top * (2 * n + 1) / 254 * 254 / (2 * top)   # (2 n + 1) / 2 of a largest magnitude 127
        rows.append(np.where(np.arange(K) % 128 == 9, 127, np.clip(t, -127, 127)))
    v = np.stack(rows)
    for e in (0, -9, 7):
        x = torch.from_numpy(v * 2.0 ** e).to(DT[xd])
        codes, scales = tern.q8_quantize(x.to(DEV), group=group)
        q, s = R.quantize(R.f64(x), np.ones(len(rows)), group)
        assert np.array_equal(codes.cpu().numpy(), q)
        equal_scales(scales.cpu(), s)
        if xd == "f32":   # products of h and w that need 64 bits: off a border by less than fp32 shows
            w = torch.from_numpy(1 + np.random.default_rng(3).integers(-2, 3, K) * 2.0 ** -23).float()
            check(x, w, 1e-6, None, group, "f32")


@pytest.mark.parametrize("xd,lo,hi", [("bf16", -120, 120), ("f32", -126, 126), ("f16", -14, 14)])
def test_values_far_from_one(xd, lo, hi):
    """Squares far beyond the fp32 range either way, without and with an epsilon."""
    rows = [R.rounded(np.random.default_rng(e + 200).standard_normal(300) * 2.0 ** e, DT[xd])
            for e in range(lo, hi + 1, 7)]
    x = torch.from_numpy(np.stack(rows)).to(DT[xd])
    for eps in (0.0, 1e-6):
        for group in (0,):
            check(x, None, eps, None, group, "f32")
    # the smallest numbers there are
    tiny = {"bf16": 2.0 ** -133, "f32": 2.0 ** -149, "f16": 2.0 ** -24}[xd]
    x = torch.from_numpy(np.random.default_rng(1).integers(-5, 6, (3, 256)) * tiny).to(DT[xd])
    check(x, None, 0.0, None, 128, "f32")


@pytest.mark.parametrize("K", [128, 384, 2304])
def test_zeros_infinities_and_nans(K):
    x = values((7, K), "bf16", K).float()
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, K - 1] = float("nan")
    x[3, 5], x[3, 6] = float("inf"), -float("inf")
    x[4, :100] = 0
    x = x.to(torch.bfloat16)
    w = torch.ones(K)
    for group in (0, 128):
        y, c, s, _ = run(x, w, 1e-6, None, group, "f32")
        _, wy, v, f = R.norm(x, w, 1e-6, None)
        got = R.f64(y)
        assert np.array_equal(np.isnan(got), np.isnan(wy))
        for row in (0, 4, 5, 6):
            R.assert_close(y[row:row + 1], wy[row:row + 1], R.norm_bound(wy[row:row + 1], torch.float32))
        q, ws = R.quantize(v, f, group)
        assert np.array_equal(c.numpy(), q)
        equal_scales(s, ws)
    assert (R.f64(y)[0] == 0).all()


def test_the_stream_may_be_written_in_place():
    x, r = values((37, 1000), "bf16", 1), values((37, 1000), "bf16", 2)
    w = values((1, 1000), "f32", 3)[0]
    y, h = tern.rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV))
    rd = r.to(DEV)
    y2 = torch.empty_like(y)
    tern.rms_norm_into(x.to(DEV), w.to(DEV), out=y2, residual=rd)
    assert torch.equal(rd, h) and torch.equal(y2, y)
    xd = x.to(DEV)
    tern.rms_norm_into(xd, w.to(DEV), out=y2, residual=r.to(DEV), residual_out=xd)
    assert torch.equal(xd, h) and torch.equal(y2, y)
    codes, scales, h2 = tern.rms_norm_q8(x.to(DEV), w.to(DEV), residual=r.to(DEV), group=0)
    assert torch.equal(h2, h)
    q, s = R.quantize(*[R.norm(x, w, 1e-6, r)[i] for i in (2, 3)], 0)
    assert np.array_equal(codes.cpu().numpy(), q)
    equal_scales(scales.cpu(), s)


def test_any_address_that_the_type_allows():
    x = values((1, 40 * 333 + 5), "bf16", 1).to(DEV)[0]
    w = values((1, 340), "f32", 2).to(DEV)[0]
    for o in range(5):
        v = x[o:o + 40 * 333].view(40, 333)
        y, c, s, _ = [t for t in run_views(v, w[o:o + 333])]
        _, wy, hv, f = R.norm(v.cpu(), w[o:o + 333].cpu(), 1e-6, None)
        R.assert_close(y, wy, R.norm_bound(wy, torch.bfloat16))
        q, ws = R.quantize(hv, f, 0)
        assert np.array_equal(c.numpy(), q)
        equal_scales(s, ws)


def run_views(v, w):
    yb = torch.zeros(40 * 333 + 3, dtype=torch.bfloat16, device=DEV)
    cb = torch.zeros(40 * 333 + 3, dtype=torch.int8, device=DEV)
    y, c = yb[3:].view(40, 333), cb[3:].view(40, 333)
    s = torch.zeros((40, 1), device=DEV)
    tern.rms_norm_into(v, w, out=y, codes=c, scales=s)
    assert (yb[:3] == 0).all() and (cb[:3] == 0).all()
    return y.cpu(), c.cpu(), s.cpu(), None


@pytest.mark.parametrize("M,K,group", [(1, 1, 0), (3, 9, 0), (5, 128, 128), (7, 1001, 0), (2, 5120, 0), (3, 5120, 128),
                                       (1, 65536, 0), (1, 131072, 128), (3000, 256, 128), (2, 20000, 0)])
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16"), ("f32", "f32")])
def test_there_and_back(M, K, group, xd, yd):
    x = values((M, K), xd, M * K)
    codes, scales = tern.q8_quantize(x.to(DEV), group=group)
    q, s = R.quantize(R.f64(x), np.ones(M), group)
    assert np.array_equal(codes.cpu().numpy(), q)
    equal_scales(scales.cpu(), s)
    y = tern.q8_dequant(codes, scales, out_dtype=DT[yd])
    want = (R.blocks(q.astype(np.float64), group) * R.f64(scales)[..., None]).reshape(M, K)
    R.assert_close(y, want, np.abs(want) * (R.STEP + R.EPS[DT[yd]] * (1 + R.STEP)) + R.TINY[DT[yd]], "dequant")


def test_sizes_of_zero():
    for M, K in ((0, 128), (3, 0), (0, 0)):
        x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
        assert tern.rms_norm(x, None).shape == (M, K)
        codes, scales = tern.rms_norm_q8(x, None, group=128)
        assert tern.q8_dequant(codes, scales).shape == (M, K)


def test_a_graph_and_another_stream():
    x, r = values((19, 5120), "bf16", 1).to(DEV), values((19, 5120), "bf16", 2).to(DEV)
    w = values((1, 5120), "bf16", 3)[0].to(DEV)
    want = tern.rms_norm_q8(x, w, residual=r, group=128)
    y = tern.rms_norm(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tern.rms_norm_q8(x, w, residual=r, group=128)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = tern.rms_norm_q8(x, w, residual=r, group=128)
        got_y = tern.rms_norm(x, w)
    for seed in (5, 6, 7):
        x.copy_(values((19, 5120), "bf16", seed))
        g.replay()
        torch.cuda.synchronize()
        want, y = tern.rms_norm_q8(x, w, residual=r, group=128), tern.rms_norm(x, w)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(got_y, y)


@pytest.mark.parametrize("M,K", [(7000, 130), (4100, 1030), (2055, 1500), (1300, 5119), (700, 9000), (530, 12800), (300, 33000)])
@pytest.mark.parametrize("xd,rd", [("bf16", "bf16"), ("f16", "f32")])
def test_rows_in_turns(M, K, xd, rd):
    """More rows than workgroups, which take the next one while they write the last; the stream in place."""
    print(f"norm M={M} K={K} {xd} {rd} in place", flush=True)
    x, r = values((M, K), xd, M + K), (values((M, K), rd, M) * 4).to(DT[rd])
    w = (values((1, K), "f32", K, 0)[0] * 0.3 + 1).to(DT[xd])
    group = 0 if K % 128 else 128
    codes, scales, h = tern.rms_norm_q8(x.to(DEV), w.to(DEV), residual=r.to(DEV), group=group)
    rd_, y = r.to(DEV), torch.empty((M, K), dtype=DT[xd], device=DEV)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    tern.rms_norm_into(x.to(DEV), w.to(DEV), out=y, codes=c2, scales=s2, residual=rd_)
    assert torch.equal(rd_, h) and torch.equal(c2, codes) and torch.equal(s2, scales)
    wh, wy, v, f = R.norm(x, w, 1e-6, r)
    assert np.array_equal(R.f64(h), wh)
    R.assert_close(y, wy, R.norm_bound(wy, DT[xd]), "norm")
    q, ws = R.quantize(v, f, group)
    assert np.array_equal(codes.cpu().numpy(), q)
    equal_scales(scales.cpu(), ws)
    if xd == rd:   # the sum into x's own buffer
        x2 = x.to(DEV)
        tern.rms_norm_into(x2, w.to(DEV), out=y, residual=r.to(DEV), residual_out=x2)
        assert torch.equal(x2, h)
