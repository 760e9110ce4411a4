"""The mixture-of-experts layer with ternary experts on the GPU: against a 64-bit
reference, bit for bit where the arithmetic is exact, its routing rules, and the
layer next to the products it is used with."""
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


class Layer:
    def __init__(self, E, H, F, seed, zeros=0.4):
        rng = np.random.default_rng(seed)
        p = [(1 - zeros) / 2, zeros, (1 - zeros) / 2]
        self.E, self.H, self.F = E, H, F
        self.gu = R.pack_ternary(rng.choice([-1, 0, 1], (E, 2 * F, H), p=p))
        self.dn = R.pack_ternary(rng.choice([-1, 0, 1], (E, H, F), p=p))
        self.gus = np.exp(rng.uniform(np.log(1e-2), np.log(1e-1), (E, 2 * F, H // 128))).astype(np.float16)
        self.ds = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), (E, H, F // 128))).astype(np.float16)
        self.d = None

    def tensors(self):
        if self.d is None:
            self.d = [dev(a) for a in (self.gu, self.gus, self.dn, self.ds)]
        return self.d

    def run(self, x, logits, k, renorm=True, yd="f32"):
        gu, gus, dn, ds = self.tensors()
        y = torch.full(x.shape, float("nan"), dtype=DT[yd], device=DEV)
        return tern.moe_into(x.to(DEV), logits.to(DEV), gu, gus, dn, ds, y, k, renorm)

    def want(self, x, logits, k, renorm, yd):
        return R.moe(R.f64(x), R.f64(logits), self.gu, self.gus, self.dn, self.ds, k, renorm, DT[yd])


def inputs(T, E, H, xd, seed, ld="f32"):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(DT[xd])
    lg = torch.from_numpy(rng.standard_normal((T, E)) * 1.5).to(DT[ld])
    return x, lg


# tokens from 1 over the chunk of 64; one expert to many; rows off every tile; K of one block up
SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 8, 1024, 512), (2, 5, 3, 640, 384), (3, 4, 4, 128, 896),
          (4, 8, 2, 2176, 256), (5, 16, 8, 384, 640), (7, 3, 1, 512, 1152), (8, 32, 4, 1280, 128), (9, 2, 2, 256, 256),
          (16, 60, 6, 512, 384), (17, 9, 5, 128, 128), (33, 100, 7, 384, 256), (64, 4, 2, 256, 128),
          (65, 6, 2, 256, 256), (130, 5, 1, 128, 256), (2, 130, 32, 128, 128), (1, 1024, 32, 128, 128),
          (1, 4, 2, 8704, 128), (6, 3, 2, 128, 8832), (4, 4, 2, 5120, 256), (3, 3, 2, 6272, 128), (2, 4, 2, 5248, 384),
          (4, 3, 1, 4096, 640)]


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
@pytest.mark.parametrize("xd,yd,ld,renorm", [("bf16", "bf16", "f32", True), ("f16", "f32", "bf16", False),
                                             ("bf16", "f32", "f16", True), ("f16", "f16", "f32", False)])
def test_layer(T, E, k, H, F, xd, yd, ld, renorm):
    print(f"moe T={T} E={E} k={k} H={H} F={F} {xd}->{yd} logits {ld}", flush=True)
    L = Layer(E, H, F, T + E + H)
    x, lg = inputs(T, E, H, xd, T * E + k, ld)
    y = L.run(x, lg, k, renorm, yd)
    want, bound = L.want(x, lg, k, renorm, yd)
    R.assert_close(y, want, bound, "moe")


@pytest.mark.parametrize("T,H,F", [(1, 16384, 128), (3, 128, 16384), (7, 16384, 128), (5, 128, 16384),
                                   (21, 7040, 128), (21, 128, 7168)])
def test_widths_at_the_limit(T, H, F):
    """Operands that fill LDS, and widths at which fewer tokens of an expert fit at a time."""
    print(f"moe T={T} H={H} F={F}", flush=True)
    L = Layer(2, H, F, T + H)
    x, lg = inputs(T, 2, H, "bf16", T + F, "f32")
    y = L.run(x, lg, 1, True, "f32")
    want, bound = L.want(x, lg, 1, True, "f32")
    R.assert_close(y, want, bound, "moe")


@pytest.mark.parametrize("T,E,H,F", [(1, 3, 256, 128), (3, 3, 1152, 256), (6, 2, 128, 384), (20, 4, 512, 128),
                                     (70, 4, 128, 256)])
@pytest.mark.parametrize("xd", ["f16", "bf16"])
def test_exact_arithmetic(T, E, H, F, xd):
    """One expert per token (weight 1), a gate of 256 (silu is the identity there), small
    integers elsewhere and power-of-two scales: every step is exact."""
    rng = np.random.default_rng(T)
    L = Layer(E, H, F, 11)
    t_up = rng.choice([-1, 0, 1], (E, F, H), p=[0.05, 0.9, 0.05])
    gate = np.zeros((E, F, H), dtype=np.int64)
    gate[:, :, 0] = 1
    L.gu = R.pack_ternary(np.concatenate([gate, t_up], axis=1))
    L.gus = np.ones((E, 2 * F, H // 128), dtype=np.float16)
    L.ds = np.exp2(rng.integers(-3, 4, (E, H, F // 128))).astype(np.float16)
    X = rng.integers(-2, 3, (T, H)).astype(np.float64)
    X[:, 0] = 256
    lg = torch.from_numpy(rng.standard_normal((T, E))).float()
    y = L.run(torch.from_numpy(X).to(DT[xd]), lg, 1)
    want = np.zeros((T, H))
    for t in range(T):
        e = int(lg[t].argmax())
        h = 256 * (X[t] @ R.dense(L.gu[e], L.gus[e])[F:].T)
        want[t] = h @ R.dense(L.dn[e], L.ds[e]).T
    assert np.array_equal(R.f64(y), want)


def test_ties_go_to_the_lowest_index():
    E, H, F = 70, 128, 128
    L = Layer(E, H, F, 3)
    x, _ = inputs(3, E, H, "bf16", 4)
    lg = torch.zeros((3, E))
    lg[1, 10:] = 1.0
    lg[2, ::3] = -0.0
    y = L.run(x, lg, 4)
    want, bound = L.want(x, lg, 4, True, "f32")
    R.assert_close(y, want, bound)


@pytest.mark.parametrize("T", [1, 3, 20, 70])
@pytest.mark.parametrize("renorm", [True, False])
def test_closed_experts_and_padding(T, renorm):
    """An expert at -inf is never taken, even where fewer than top_k are open; a token with all
    of them closed gets zeros, whatever its row of x holds."""
    E, H, F, k = 6, 256, 128, 3
    L = Layer(E, H, F, 5)
    x, lg = inputs(T, E, H, "f16", 6)
    lg[:, 1] = -float("inf")
    lg[0, :] = -float("inf")
    lg[0, 4] = 0.5
    clean = L.run(x, lg, k, renorm)
    want, bound = L.want(x, lg, k, renorm, "f32")
    R.assert_close(clean, want, bound)
    lg[T - 1] = -float("inf")
    x[T - 1] = float("nan")
    y = L.run(x, lg, k, renorm)
    assert (y[T - 1] == 0).all()
    R.assert_close(y[:T - 1], want[:T - 1], bound[:T - 1])


@pytest.mark.parametrize("T", [2, 5, 20, 70])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["x", "logits"])
def test_non_finite_values_stay_in_their_token(T, bad, where):
    E, H, F, k = 4, 256, 256, 2
    L = Layer(E, H, F, 7, zeros=0.1)
    x, lg = inputs(T, E, H, "bf16", 8)
    want, bound = L.want(x, lg, k, True, "f32")
    if where == "x":
        x[T // 2, 3] = bad
    else:
        lg[T // 2, 1] = bad
    y = L.run(x, lg, k)
    keep = [t for t in range(T) if t != T // 2]
    R.assert_close(y[keep], want[keep], bound[keep])
    assert torch.isnan(y[T // 2]).all()


@pytest.mark.parametrize("T", [1, 4, 30])
def test_all_tokens_on_one_expert(T):
    E, H, F = 7, 384, 256
    L = Layer(E, H, F, 9)
    x, lg = inputs(T, E, H, "bf16", 10)
    lg[:, 5] += 100
    y = L.run(x, lg, 1)
    want, bound = L.want(x, lg, 1, True, "f32")
    R.assert_close(y, want, bound)


@pytest.mark.parametrize("T", [1, 3, 12, 66])
def test_repeated_calls_agree_bit_for_bit_and_leave_neighbours(T):
    E, H, F, k = 12, 640, 384, 4
    L = Layer(E, H, F, 12)
    x, lg = inputs(T, E, H, "bf16", 13)
    first = L.run(x, lg, k, yd="bf16")
    buf = torch.full((T + 2, H), 5.0, dtype=torch.bfloat16, device=DEV)
    gu, gus, dn, ds = L.tensors()
    for _ in range(3):
        tern.moe_into(x.to(DEV), lg.to(DEV), gu, gus, dn, ds, buf[1:T + 1], k)
        assert torch.equal(buf[1:T + 1], first)
    assert (buf[0] == 5).all() and (buf[T + 1] == 5).all()


@pytest.mark.parametrize("T", [1, 3, 24])
def test_streams_and_graph_replays(T):
    """Two captured graphs and two streams at once, each call with a workspace of its own;
    replays on new inputs with eager work between them."""
    E, H, F, k = 16, 512, 256, 4
    L = Layer(E, H, F, 14)
    gu, gus, dn, ds = L.tensors()
    data = [tuple(t.to(DEV) for t in inputs(T, E, H, "bf16", 20 + i)) for i in range(4)]
    want = [tern.moe(x, lg, gu, gus, dn, ds, k) for x, lg in data]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):
        a = tern.moe(*data[0], gu, gus, dn, ds, k)
        with torch.cuda.stream(side):
            b = tern.moe(*data[1], gu, gus, dn, ds, k)
        outs.append((a, b))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    graphs = []
    for i in range(2):
        x, lg = data[i][0].clone(), data[i][1].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = tern.moe(x, lg, gu, gus, dn, ds, k)
        graphs.append((g, x, lg, y))
    for i in (2, 3, 1, 0):
        for j, (g, x, lg, y) in enumerate(graphs):
            x.copy_(data[(i + j) % 4][0])
            lg.copy_(data[(i + j) % 4][1])
            g.replay()
        with torch.cuda.stream(side):
            tern.moe(*data[0], gu, gus, dn, ds, k)
        torch.cuda.synchronize()
        for j, (g, x, lg, y) in enumerate(graphs):
            assert torch.equal(y, want[(i + j) % 4])


@pytest.mark.parametrize("T", [1, 6])
def test_experts_past_32_bits(T):
    """The last of 40 experts, whose rows start 5 GB into the weights, gives the bits it gives alone."""
    E, H, F = 40, 16384, 16384
    print(f"moe T={T} E={E} H={H} F={F}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(T)
    codes = [torch.zeros((E, 2 * F, H // 4), dtype=torch.uint8, device=DEV),
             torch.zeros((E, H, F // 4), dtype=torch.uint8, device=DEV)]
    scales = [torch.zeros((E, 2 * F, H // 128), dtype=torch.float16, device=DEV),
              torch.zeros((E, H, F // 128), dtype=torch.float16, device=DEV)]
    for c, s in zip(codes, scales):
        c[-1].copy_(torch.randint(0, 256, c[-1].shape, dtype=torch.uint8, device=DEV, generator=g))
        s[-1].fill_(2.0 ** -7)
    x = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    lg = torch.full((T, E), -float("inf"), device=DEV)
    lg[:, -1] = 0.5
    y = tern.moe(x, lg, codes[0], scales[0], codes[1], scales[1], 1, out_dtype=torch.float32)
    one = tern.moe(x, lg[:, -1:].contiguous(), codes[0][-1:].contiguous(), scales[0][-1:].contiguous(),
                   codes[1][-1:].contiguous(), scales[1][-1:].contiguous(), 1, out_dtype=torch.float32)
    assert torch.isfinite(y).all() and y.abs().max() > 0
    assert torch.equal(y, one)


def test_refusals():
    E, H, F = 4, 256, 128
    L = Layer(E, H, F, 15)
    gu, gus, dn, ds = L.tensors()
    x, lg = (t.to(DEV) for t in inputs(2, E, H, "bf16", 16))
    with pytest.raises(tern.TernError):
        tern.moe(x, lg, gu, gus, dn, ds, 0)
    with pytest.raises(tern.TernError):
        tern.moe(x, lg, gu, gus, dn, ds, 5)
    with pytest.raises(ValueError):
        tern.moe(x, lg[:, :3].contiguous(), gu, gus, dn, ds, 2)
    with pytest.raises(ValueError):
        tern.moe(x, lg, gu[:3], gus, dn, ds, 2)
    with pytest.raises(ValueError):
        tern.moe(x, lg, gu, gus, dn.transpose(1, 2), ds, 2)
    with pytest.raises(TypeError):
        tern.moe(x.float(), lg, gu, gus, dn, ds, 2)
    with pytest.raises(ValueError):
        tern.moe(x, lg.cpu(), gu, gus, dn, ds, 2)
    assert tern.moe(x[:0], lg[:0], gu, gus, dn, ds, 2).shape == (0, H)


@pytest.mark.parametrize("T", [1, 4, 40])
def test_block_of_a_decoder(T):
    """The operators together, as a mixed-precision decoder block uses them: a 4-bit projection,
    a 4-bit router whose fp32 outputs are the logits, the experts, and a 4-bit head on quantised
    activations; against the 64-bit reference of each step on the step's own inputs."""
    E, H, F, k, V = 16, 512, 256, 4, 300
    rng = np.random.default_rng(T)
    L = Layer(E, H, F, 17)
    gu, gus, dn, ds = L.tensors()

    def quantised(n):
        return tern.mx_quantize(torch.from_numpy(rng.standard_normal((n, H)) / np.sqrt(H)).float().to(DEV))

    def check_product(y, x, w, dt):
        W = R.values(w[0].cpu().numpy(), w[1].cpu().numpy())
        want = R.f64(x) @ W.T
        R.assert_close(y, want, R.product_bound(R.f64(x), W, want, dt))

    proj, router, head = quantised(H), quantised(E), quantised(V)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).to(DEV)
    a = tern.mx_matmul(x, *proj)
    check_product(a, x, proj, torch.bfloat16)
    lg = tern.mx_matmul(a, *router, out_dtype=torch.float32)
    check_product(lg, a, router, torch.float32)
    y = tern.moe(a, lg, gu, gus, dn, ds, k)
    want, bound = L.want(a, lg, k, True, "bf16")
    R.assert_close(y, want, bound)
    q = tern.mx_quantize(y)
    z = tern.mx_matmul_mx(*q, *head, out_dtype=torch.float32)
    check_product(z, tern.mx_dequant(*q), head, torch.float32)
