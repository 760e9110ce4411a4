"""Routing on the GPU, against a 64-bit reference, and the expert layer that takes its
experts and weights as given."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mx_util as X  # noqa: E402
import q8_util as R  # noqa: E402

tern = pytest.importorskip("ternary_weight_matmul_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(logits, top_k, score="softmax", bias=None, groups=1, keep=1, best=1, renorm=True, scale=1.0):
    ids, w = tern.moe_route(logits.to(DEV), top_k, score=score, bias=bias.to(DEV) if bias is not None else None,
                            groups=groups, keep_groups=keep, group_best=best, renormalize=renorm, scale=scale)
    want_ids, want_w = R.route(R.f64(logits), top_k, score, R.f64(bias) if bias is not None else None, groups, keep, best,
                               renorm, float(np.float32(scale)))
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = R.f64(w)
    # 64 bits, rounded once to fp32
    ok = (np.isnan(got) & np.isnan(want_w)) | (np.abs(got - want_w) <= np.abs(want_w) * R.STEP * 1.001 + 2.0 ** -149)
    assert ok.all(), (got[~ok][:4], want_w[~ok][:4])
    return ids, w


# E, top_k, groups, kept ones: one expert to the most; groups of odd sizes and numbers
CASES = [(1, 1, 1, 1), (2, 2, 1, 1), (5, 3, 1, 1), (8, 2, 2, 1), (60, 4, 6, 2), (63, 6, 7, 3), (64, 8, 1, 1), (64, 8, 8, 4),
         (65, 8, 5, 5), (96, 6, 3, 2), (128, 8, 1, 1), (129, 9, 43, 7), (160, 6, 8, 3), (256, 8, 8, 4), (256, 32, 64, 9),
         (257, 10, 1, 1), (384, 8, 1, 1), (512, 22, 16, 7), (1000, 7, 10, 10), (1024, 32, 64, 33)]


@pytest.mark.parametrize("E,top_k,groups,keep", CASES)
@pytest.mark.parametrize("score,biased,best,renorm,ld", [("softmax", False, 1, True, "f32"), ("sigmoid", True, 2, True, "f32"),
                                                         ("softmax", True, 1, False, "bf16"), ("sigmoid", False, 1, False, "f16"),
                                                         ("sigmoid", False, 2, True, "f32"), ("softmax", False, 1, False, "bf16")])
def test_route(E, top_k, groups, keep, score, biased, best, renorm, ld):
    best = min(best, E // groups)
    print(f"route E={E} k={top_k} groups {keep}/{groups} {score} bias {biased} best {best} {ld}", flush=True)
    rng = np.random.default_rng(E + top_k)
    lg = torch.from_numpy(rng.standard_normal((9, E)) * 2).to(DT[ld])
    bias = torch.from_numpy(rng.standard_normal(E) * 0.1).float() if biased else None
    check(lg, top_k, score, bias, groups, keep, best, renorm, 2.5 if renorm else 1.0)


@pytest.mark.parametrize("T", [1, 3, 4, 5, 700, 9000])
def test_numbers_of_tokens(T):
    rng = np.random.default_rng(T)
    lg = torch.from_numpy(rng.standard_normal((T, 64))).float()
    b = torch.from_numpy(rng.standard_normal(64) * 0.05).float()
    rows = min(T, 300)
    ids, w = tern.moe_route(lg.to(DEV), 6, score="sigmoid", bias=b.to(DEV), groups=4, keep_groups=2, group_best=2)
    for sl in (slice(0, rows), slice(T - rows, T)):
        want_ids, want_w = R.route(R.f64(lg)[sl], 6, "sigmoid", R.f64(b), 4, 2, 2, True, 1.0)
        assert np.array_equal(ids.cpu().numpy()[sl], want_ids)
        assert (np.abs(R.f64(w)[sl] - want_w) <= want_w * R.STEP * 1.001).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score):
    lg = torch.zeros((5, 96))
    lg[1, 10:] = 1.0
    lg[2, ::3] = -0.0
    lg[3] = torch.arange(96) % 4
    check(lg, 7, score)
    check(lg, 7, score, groups=4, keep=2)
    check(lg, 7, score, bias=torch.zeros(96), groups=4, keep=2, best=2)
    # equal sums of a score and a bias only where both are equal
    check(lg, 7, score, bias=(torch.arange(96) % 5).float() * 0.25, groups=8, keep=3, best=2)


def test_choices_that_hang_on_the_last_bits():
    """Scores that fp32 cannot tell apart, in an order against the index's."""
    E = 64
    lg = (20 + torch.arange(E).float() * 2.0 ** -10)[None].repeat(2, 1)   # sigmoids next to 1
    check(lg, 8, "sigmoid", bias=torch.zeros(E))
    check(lg, 8, "sigmoid", groups=8, keep=2, best=2)
    check(torch.full((1, E), 0.3) + torch.arange(E) * 2.0 ** -24, 8, "sigmoid", bias=torch.full((E,), 100.0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_closed_experts_infinities_and_nans(score, biased, groups, keep, best):
    E = 32
    rng = np.random.default_rng(5)
    lg = torch.from_numpy(rng.standard_normal((8, E))).float()
    lg[0] = -INF                 # padding: no expert at all
    lg[1, :] = -INF
    lg[1, 30] = 0.5              # a single one
    lg[2, 8:24] = -INF           # whole groups
    lg[3, 3] = INF
    lg[4] = torch.finfo(torch.float32).min
    lg[5, 1:9] = -INF
    lg[6, 7] = torch.finfo(torch.float32).max
    bias = torch.from_numpy(rng.standard_normal(E) * 0.1).float() if biased else None
    if score == "softmax" and biased:
        lg[3, 3] = 1.0           # with a bias every score of such a row is NaN: the lowest indices
    check(lg, 8, score, bias, groups, keep, best)
    nan = lg.clone()
    nan[7, 11] = float("nan")
    if not (score == "softmax" and biased) and not (score == "softmax" and best == 2):
        check(nan, 8, score, bias, groups, keep, best)
    if biased:
        bias[5], bias[9] = -INF, INF
        check(lg, 8, score, bias, groups, keep, best)


def test_far_logits():
    """Weights where fp32 exponentials would be 0 or infinite."""
    lg = torch.tensor([[-200.0, -210.0, -400.0, -700.0], [300.0, 290.0, -800.0, 100.0], [-3e4, -3e4, -3.1e4, -2.9e4]])
    check(lg, 3, "sigmoid", renorm=True)
    check(lg, 3, "sigmoid", renorm=False)
    check(lg, 4, "softmax", renorm=True)
    check(lg, 4, "softmax", renorm=False)


# ---- the layer --------------------------------------------------------------------

class Layer:
    def __init__(self, E, H, F, seed):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.F = E, H, F
        self.gu = R.pack_ternary(rng.choice([-1, 0, 1], (E, 2 * F, H), p=[0.3, 0.4, 0.3]))
        self.dn = R.pack_ternary(rng.choice([-1, 0, 1], (E, H, F), p=[0.3, 0.4, 0.3]))
        self.gus = np.exp(rng.uniform(np.log(1e-2), np.log(1e-1), (E, 2 * F, H // 128))).astype(np.float16)
        self.ds = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), (E, H, F // 128))).astype(np.float16)
        self.d = [torch.from_numpy(a).to(DEV) for a in (self.gu, self.gus, self.dn, self.ds)]

    def run(self, x, ids, w, yd):
        y = torch.full(x.shape, float("nan"), dtype=DT[yd], device=DEV)
        return tern.moe_routed_into(x.to(DEV), ids.to(DEV), w.to(DEV), *self.d, y)

    def want(self, x, ids, w, yd):
        """The layer in 64 bits for given experts: the reference of the layer that routes by itself, with
        logits that open exactly a token's experts and its weights put in by linearity."""
        xs, idn, wn = R.f64(x), ids.cpu().numpy(), R.f64(w)
        T = xs.shape[0]
        y, bound = np.zeros((T, self.H)), np.zeros((T, self.H))
        for j in range(idn.shape[1]):
            rows = np.where((idn[:, j] >= 0) & (idn[:, j] < self.E))[0]
            if rows.size == 0:
                continue
            lg = np.full((rows.size, self.E), -np.inf)
            lg[np.arange(rows.size), idn[rows, j]] = 0.0
            part, b = X.moe(xs[rows], lg, self.gu, self.gus, self.dn, self.ds, 1, True, torch.float32)
            y[rows] += wn[rows, j:j + 1] * part
            bound[rows] += np.abs(wn[rows, j:j + 1]) * b * (1 + 2.0 ** -20)
        bound += idn.shape[1] * 2.0 ** -23 * (np.abs(y) + bound)
        return y, bound + R.EPS[DT[yd]] * (np.abs(y) + bound) + R.TINY[DT[yd]]


@pytest.mark.parametrize("T,E,k,H,F", [(1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 6, 1024, 512), (2, 5, 3, 640, 384),
                                       (3, 4, 4, 128, 896), (4, 8, 2, 2176, 256), (5, 16, 8, 384, 640), (9, 2, 2, 256, 256),
                                       (17, 9, 5, 128, 128), (64, 4, 2, 256, 128), (65, 6, 2, 256, 256), (130, 5, 1, 128, 256)])
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f16", "f32")])
def test_routed_layer(T, E, k, H, F, xd, yd):
    print(f"routed T={T} E={E} k={k} H={H} F={F} {xd}->{yd}", flush=True)
    L = Layer(E, H, F, T + E)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(DT[xd])
    lg = torch.from_numpy(rng.standard_normal((T, E))).float().to(DEV)
    b = torch.from_numpy(rng.standard_normal(E) * 0.1).float().to(DEV)
    ids, w = tern.moe_route(lg, k, score="sigmoid", bias=b, scale=2.5)
    want, bound = L.want(x, ids, w, yd)
    R.assert_close(L.run(x, ids, w, yd), want, bound, "routed layer")


@pytest.mark.parametrize("T", [1, 2, 4, 5, 70])
def test_the_same_expert_twice_and_none(T):
    E, H, F, k = 6, 256, 256, 5
    L = Layer(E, H, F, 3)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16)
    ids = torch.from_numpy(rng.integers(-2, E + 2, (T, k)).astype(np.int32))
    w = torch.from_numpy(rng.standard_normal((T, k))).float()
    ids[0] = torch.tensor([2, 2, -1, 2, 4], dtype=torch.int32)
    if T > 1:
        ids[1] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31, -7], dtype=torch.int32)
        w[1] = float("nan")     # nothing takes them
    want, bound = L.want(x, ids, torch.where((ids >= 0) & (ids < E), w, 0.0), "f32")
    y = L.run(x, ids, w, "f32")
    R.assert_close(y, want, bound, "twice")
    if T > 1:
        assert (y[1] == 0).all()


@pytest.mark.parametrize("T", [1, 3, 20, 70])
def test_agrees_with_the_layer_that_routes_by_itself(T):
    E, H, F, k = 16, 512, 384, 4
    L = Layer(E, H, F, 9)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16)
    lg = torch.from_numpy(rng.standard_normal((T, E))).float()
    lg[0] = -INF
    ids, w = tern.moe_route(lg.to(DEV), k)
    assert (ids[0] == -1).all() and (w[0] == 0).all()
    y = L.run(x, ids, w, "f32")
    own = tern.moe(x.to(DEV), lg.to(DEV), *L.d, top_k=k, out_dtype=torch.float32)
    want, bound = L.want(x, ids, w, "f32")
    R.assert_close(y, want, bound)
    assert (np.abs(R.f64(own) - want) <= bound * 1.01 + 2.0 ** -20 * np.abs(want)).all()
    assert (y[0] == 0).all()


@pytest.mark.parametrize("T", [1, 30])
def test_a_layer_from_the_stream_on_in_a_graph(T):
    """Norm, router, routing and experts, as a decode step runs them: captured, replayed on other
    tokens, against the same calls outside of a graph."""
    E, H, F, k = 16, 512, 256, 4
    L = Layer(E, H, F, 2)
    rng = np.random.default_rng(T)
    stream = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).to(DEV)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).to(DEV)
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(H)).float().to(DEV)
    router = R.pack_ternary(rng.choice([-1, 0, 1], (E, H)))
    router, rs = torch.from_numpy(router).to(DEV), torch.full((E, H // 128), 0.1, dtype=torch.float16, device=DEV)
    bias = torch.from_numpy(rng.standard_normal(E) * 0.1).float().to(DEV)

    def layer():
        y, h = tern.rms_norm(x, w, residual=stream)
        codes, scales = tern.q8_quantize(y)
        lg = tern.matmul_q8(codes, scales, router, rs, out_dtype=torch.float32)
        ids, ww = tern.moe_route(lg, k, score="sigmoid", bias=bias, groups=4, keep_groups=2, group_best=2, scale=2.5)
        return h, ids, ww, tern.moe_routed(y, ids, ww, *L.d)

    layer()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer()
    for seed in (1, 2, 3):
        x.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((T, H))))
        g.replay()
        torch.cuda.synchronize()
        want = layer()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        xs = R.f64(tern.rms_norm(x, w, residual=stream)[0])
        ref, bound = L.want(torch.from_numpy(xs), got[1], got[2], "bf16")
        R.assert_close(got[3], ref, bound)
