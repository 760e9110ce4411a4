"""The C entry points of the microscaled and mixture-of-experts operators on the
CPU: refusals before anything is launched, and the binding's own checks."""
import pytest

torch = pytest.importorskip("torch")
tern = pytest.importorskip("ternary_weight_matmul_amd", reason="libtern.so not built")
L = tern.lib

OK, NULL, SHAPE, GROUP, DTYPE, ALIGN, UNSUP = 0, 1, 2, 3, 4, 5, 6
F16, BF16, F32 = 0, 1, 2
P = 4096   # a fake, aligned, non-NULL device address; never dereferenced


def quant(X=P, xd=BF16, C=P, S=P, M=4, K=64):
    return L.tern_mx_quantize(X, xd, C, S, M, K, None)


def dequant(X=P, xd=BF16, C=P, S=P, M=4, K=64):
    return L.tern_mx_dequant(C, S, X, xd, M, K, None)


@pytest.mark.parametrize("f", [quant, dequant])
@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(K=-32), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=(1 << 30) + 32), SHAPE),
    (dict(K=48), GROUP), (dict(K=4), GROUP), (dict(xd=3), DTYPE),
    (dict(X=0), NULL), (dict(C=0), NULL), (dict(S=0), NULL),
    (dict(X=P + 8), ALIGN), (dict(C=P + 4), ALIGN),
    (dict(M=0, X=0, C=0, S=0), OK), (dict(K=0, X=0, C=0, S=0), OK),
])
def test_mx_convert_rejects(f, kw, want):
    assert f(**kw) == want


def mm(X=P, xd=BF16, W=P, S=P, Y=P, yd=BF16, M=2, N=16, K=64):
    return L.tern_mx_matmul(X, xd, W, S, Y, yd, M, N, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-32), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(K=(1 << 30) + 32), SHAPE), (dict(K=(1 << 24) + 32), SHAPE), (dict(K=40), GROUP), (dict(xd=F32), DTYPE), (dict(xd=9), DTYPE),
    (dict(yd=5), DTYPE), (dict(X=0), NULL), (dict(W=0), NULL), (dict(S=0), NULL), (dict(Y=0), NULL),
    (dict(K=0, Y=0), NULL), (dict(X=P + 2), ALIGN), (dict(W=P + 8), ALIGN), (dict(Y=P + 1), ALIGN),
    (dict(Y=P + 2, yd=F32), ALIGN), (dict(M=0, X=0, W=0, S=0, Y=0), OK), (dict(N=0, X=0, W=0, S=0, Y=0), OK),
])
def test_mx_matmul_rejects(kw, want):
    assert mm(**kw) == want


def mmx(X=P, XS=P, W=P, S=P, Y=P, yd=BF16, M=2, N=16, K=64):
    return L.tern_mx_matmul_mx(X, XS, W, S, Y, yd, M, N, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(K=(1 << 24) + 32), SHAPE), (dict(K=40), GROUP), (dict(yd=5), DTYPE), (dict(X=0), NULL),
    (dict(XS=0), NULL),
    (dict(W=0), NULL), (dict(S=0), NULL), (dict(Y=0), NULL), (dict(X=P + 8), ALIGN), (dict(W=P + 8), ALIGN),
    (dict(M=0, X=0, XS=0, W=0, S=0, Y=0), OK),
])
def test_mx_matmul_mx_rejects(kw, want):
    assert mmx(**kw) == want


def moe(X=P, xd=BF16, lg=P, ld=F32, gu=P, gus=P, dn=P, ds=P, Y=P, yd=BF16, T=2, E=8, k=2, H=256, F=128, G=128,
        rn=1, ws=P, wb=1 << 40):
    return L.tern_moe(X, xd, lg, ld, gu, gus, dn, ds, Y, yd, T, E, k, H, F, G, rn, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(E=-1), SHAPE), (dict(H=-128), SHAPE), (dict(F=-128), SHAPE), (dict(k=0), SHAPE),
    (dict(k=9), SHAPE), (dict(E=0, k=1), SHAPE), (dict(H=(1 << 30) + 128), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(H=16384 + 128), SHAPE), (dict(F=16384 + 128), SHAPE),
    (dict(H=192), GROUP), (dict(F=64), GROUP), (dict(G=0), GROUP), (dict(G=-128), GROUP),
    (dict(G=64), UNSUP), (dict(E=1025), UNSUP), (dict(E=64, k=33), UNSUP),
    (dict(xd=F32), DTYPE), (dict(ld=4), DTYPE), (dict(yd=4), DTYPE),
    (dict(X=0), NULL), (dict(lg=0), NULL), (dict(gu=0), NULL), (dict(gus=0), NULL), (dict(dn=0), NULL),
    (dict(ds=0), NULL), (dict(Y=0), NULL), (dict(ws=0), NULL),
    (dict(X=P + 8), ALIGN), (dict(lg=P + 2), ALIGN), (dict(gu=P + 8), ALIGN), (dict(gus=P + 1), ALIGN),
    (dict(dn=P + 8), ALIGN), (dict(ds=P + 1), ALIGN), (dict(Y=P + 1), ALIGN), (dict(ws=P + 128), ALIGN),
    (dict(wb=0), SHAPE), (dict(T=0, X=0, lg=0, Y=0, ws=0), OK),
])
def test_moe_rejects(kw, want):
    assert moe(**kw) == want


def test_moe_workspace():
    need = L.tern_moe_workspace(2, 8, 2, 256, 128)
    assert need > 0
    assert moe(wb=need - 1) == SHAPE
    # a call's tokens are taken 64 at a time: its workspace stops growing there
    assert L.tern_moe_workspace(64, 8, 2, 256, 128) == L.tern_moe_workspace(1000, 8, 2, 256, 128)
    assert L.tern_moe_workspace(-1, 8, 2, 256, 128) == 0
    assert L.tern_moe_workspace(0, 8, 2, 256, 128) == 0


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    codes, exps = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError):
        tern.mx_quantize(x)
    with pytest.raises(ValueError):
        tern.mx_dequant(codes, exps)
    with pytest.raises(ValueError):
        tern.mx_matmul(x, codes, exps)
    with pytest.raises(ValueError):
        tern.mx_matmul_mx(codes, exps, codes, exps)
    with pytest.raises(TypeError):
        tern.mx_quantize(x.double())
    with pytest.raises(TypeError):
        tern.mx_matmul(x.float(), codes, exps)
    with pytest.raises(ValueError):
        tern.moe(x, torch.zeros((2, 4)), codes[None], exps[None].half(), codes[None], exps[None].half(), 1)
