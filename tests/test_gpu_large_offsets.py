"""Matrices of more than 2^31 elements through the norm, the 8-bit activations, their product and
the routing: the last rows are those of a small call."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

tern = pytest.importorskip("ternary_weight_matmul_amd")

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def values(M, K, dtype=torch.bfloat16):
    """Rows that differ, made in place."""
    x = torch.empty((M, K), dtype=dtype, device=DEV)
    return x.normal_(generator=torch.Generator(device=DEV).manual_seed(M))


def same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("M,K", [(430001, 5121), (16800001, 128), (33001, 65536)])
def test_norm_and_codes(M, K):
    print(f"norm M={M} K={K}", flush=True)
    x = values(M, K)
    w = torch.linspace(0.5, 1.5, K, device=DEV)
    tail = x[-7:].clone()
    group = 128 if K % 128 == 0 else 0
    same((tern.rms_norm(x, w)[-7:],), (tern.rms_norm(tail, w),))
    r = x.clone()
    codes, scales = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty((M, K // 128 if group else 1), device=DEV)
    tern.rms_norm_into(x, w, codes=codes, scales=scales, residual=r)
    same((codes[-7:], scales[-7:], r[-7:]), tern.rms_norm_q8(tail, w, residual=tail, group=group))
    del r
    same((tern.q8_dequant(codes, scales, out_dtype=torch.bfloat16)[-7:],), (tern.q8_dequant(codes[-7:], scales[-7:], out_dtype=torch.bfloat16),))
    codes, scales = tern.q8_quantize(x, group=group)
    same((codes[-7:], scales[-7:]), tern.q8_quantize(tail, group=group))


@pytest.mark.parametrize("M,N,K", [(66001, 33000, 128), (66001, 33000, 512), (40, 54000001, 128), (40, 54000001, 512), (8, 1 << 28, 128),
                                   (9, 250000001, 512)])
@pytest.mark.parametrize("group", [0, 128])
def test_product(M, N, K, group):
    print(f"matmul_q8 M={M} N={N} K={K} group={group}", flush=True)
    q = torch.randint(-128, 128, (M, K), dtype=torch.int8, device=DEV)
    xs = torch.rand((M, K // 128 if group else 1), device=DEV).exp2_()
    packed = torch.randint(0, 256, (N, K // 4), dtype=torch.uint8, device=DEV)
    ws = torch.rand((N, K // 128), dtype=torch.float16, device=DEV)
    y = tern.matmul_q8(q, xs, packed, ws)
    # one rounding to bf16 of sums that differ in their order: the last rows and columns, and some in between
    rows = torch.unique(torch.tensor([0, M // 2, M - 2, M - 1], device=DEV))
    for cols in (slice(N - 333, N), slice(N // 2, N // 2 + 100), slice(0, 100)):
        t = torch.stack([(packed[cols] >> (2 * i)) & 3 for i in range(4)], -1).reshape(-1, K)
        t = (t == 1).double() - (t == 2).double()
        x = q[rows].double().view(len(rows), K // 128, 128) * xs[rows].double().view(len(rows), -1, 1)
        want = x.view(len(rows), K) @ (t.view(-1, K // 128, 128) * ws[cols].double().unsqueeze(-1)).view(-1, K).t().contiguous()
        scale = x.abs().view(len(rows), K) @ (t.abs().view(-1, K // 128, 128) * ws[cols].double().unsqueeze(-1)).view(-1, K).t().contiguous()
        got = y[rows][:, cols].double()
        bound = (K // 128 + 8) * 2.0 ** -24 * scale
        assert ((got - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all()


def test_routing():
    T, E = 2100001, 1024
    lg = values(T, E)
    bias = torch.linspace(-0.1, 0.1, E, device=DEV)
    for kw in (dict(), dict(score="sigmoid", bias=bias, groups=8, keep_groups=3, group_best=2)):
        ids, w = tern.moe_route(lg, 8, **kw)
        same((ids[-5:], w[-5:]), tern.moe_route(lg[-5:].clone(), 8, **kw))
