"""The C entry points of the norm, the 8-bit activations and the routing on the CPU:
refusals before anything is launched, and the binding's own checks."""
import pytest

torch = pytest.importorskip("torch")
tern = pytest.importorskip("ternary_weight_matmul_amd", reason="libtern.so not built")
L = tern.lib

OK, NULL, SHAPE, GROUP, DTYPE, ALIGN, UNSUP = 0, 1, 2, 3, 4, 5, 6
F16, BF16, F32 = 0, 1, 2
P = 4096   # a fake, aligned, non-NULL device address; never dereferenced
INF, NAN = float("inf"), float("nan")


def norm(X=P, xd=BF16, r=0, rd=BF16, w=P, wd=F32, h=0, Y=P, yd=BF16, C=0, S=0, g=0, M=4, K=256, eps=1e-6):
    return L.tern_rms_norm(X, xd, r, rd, w, wd, h, Y, yd, C, S, g, M, K, eps, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(K=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=65537), SHAPE),
    (dict(xd=3), DTYPE), (dict(wd=7), DTYPE), (dict(yd=-1), DTYPE), (dict(r=P, h=P, rd=F16), DTYPE),
    (dict(r=P, h=P, xd=F32, rd=BF16), DTYPE), (dict(X=0), NULL), (dict(Y=0), NULL), (dict(r=P), NULL),
    (dict(h=P), NULL), (dict(C=P), NULL), (dict(S=P), NULL),
    (dict(C=P, S=P, g=64), UNSUP), (dict(C=P, S=P, g=-1), UNSUP), (dict(C=P, S=P, g=128, K=200), GROUP),
    (dict(eps=-1.0), UNSUP), (dict(eps=INF), UNSUP), (dict(eps=NAN), UNSUP),
    (dict(X=P + 1), ALIGN), (dict(Y=P + 1), ALIGN), (dict(w=P + 2), ALIGN), (dict(r=P + 1, h=P), ALIGN),
    (dict(r=P, h=P + 2, rd=F32), ALIGN), (dict(C=P, S=P + 2), ALIGN), (dict(Y=P + 2, yd=F32), ALIGN),
    (dict(M=0, X=0, Y=0, w=0), OK), (dict(K=0, X=0, Y=0, w=0), OK),
])
def test_rms_norm_rejects(kw, want):
    assert norm(**kw) == want


def quant(D=P, d=BF16, C=P, S=P, g=0, M=4, K=256):
    return L.tern_q8_quantize(D, d, C, S, g, M, K, None)


def dequant(D=P, d=BF16, C=P, S=P, g=0, M=4, K=256):
    return L.tern_q8_dequant(C, S, g, D, d, M, K, None)


@pytest.mark.parametrize("f", [quant, dequant])
@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(K=-128), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=(1 << 30) + 128), SHAPE),
    (dict(g=32), UNSUP), (dict(g=128, K=100), GROUP), (dict(d=3), DTYPE), (dict(D=0), NULL), (dict(C=0), NULL),
    (dict(S=0), NULL), (dict(D=P + 1), ALIGN), (dict(S=P + 2), ALIGN), (dict(M=0, D=0, C=0, S=0), OK),
    (dict(K=0, D=0, C=0, S=0), OK),
])
def test_q8_convert_rejects(f, kw, want):
    assert f(**kw) == want


def test_a_row_that_is_too_long_for_one_scale():
    assert quant(K=65537) == SHAPE


def mm(C=P, XS=P, qg=0, W=P, S=P, Y=P, yd=BF16, M=2, N=16, K=256, G=128, ws=0, wb=0):
    return L.tern_matmul_q8(C, XS, qg, W, S, Y, yd, M, N, K, G, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-128), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(K=(1 << 23) + 128), SHAPE), (dict(M=(1 << 28) + 1), SHAPE), (dict(N=(1 << 28) + 1), SHAPE),
    (dict(M=1 << 20, N=(1 << 16) + 1), SHAPE), (dict(K=200), GROUP), (dict(G=0), GROUP), (dict(G=-128), GROUP), (dict(G=64), UNSUP),
    (dict(qg=64), UNSUP), (dict(qg=-128), UNSUP), (dict(yd=3), DTYPE), (dict(C=0), NULL), (dict(XS=0), NULL),
    (dict(W=0), NULL), (dict(S=0), NULL), (dict(Y=0), NULL), (dict(K=0, Y=0), NULL), (dict(C=P + 8), ALIGN),
    (dict(XS=P + 2), ALIGN), (dict(W=P + 8), ALIGN), (dict(S=P + 1), ALIGN), (dict(Y=P + 1), ALIGN),
    (dict(Y=P + 2, yd=F32), ALIGN), (dict(M=0, C=0, XS=0, W=0, S=0, Y=0), OK), (dict(N=0, C=0, XS=0, W=0, S=0, Y=0), OK),
])
def test_matmul_q8_rejects(kw, want):
    assert mm(**kw) == want


def test_matmul_q8_workspace():
    assert L.tern_matmul_q8_workspace(4, 16, 256) == 0
    big = dict(M=1100, N=7501, K=2816)
    need = L.tern_matmul_q8_workspace(*big.values())
    assert need >= 1100 * 2816 * 3 // 2
    assert mm(**big) == NULL
    assert mm(**big, ws=P, wb=need - 1) == SHAPE
    assert mm(**big, ws=P + 8, wb=need) == ALIGN
    for bad in ((-1, 4, 128), (300, -4, 128), (300, 64, -128), (300, 64, 100), (0, 64, 128), (300, 0, 128), (300, 64, 0),
                ((1 << 28) + 1, 64, 128), (300, (1 << 28) + 1, 128), (1 << 20, (1 << 16) + 1, 128)):
        assert L.tern_matmul_q8_workspace(*bad) == 0


def route(lg=P, ld=F32, b=P, i=P, w=P, T=2, E=64, k=8, sc=1, g=8, kg=4, best=2, rn=1, f=1.0):
    return L.tern_moe_route(lg, ld, b, i, w, T, E, k, sc, g, kg, best, rn, f, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=-8), SHAPE), (dict(T=1 << 31), SHAPE), (dict(k=0), SHAPE),
    (dict(k=33, E=32, g=1, kg=1), SHAPE), (dict(k=17, kg=2), SHAPE), (dict(kg=0), SHAPE), (dict(kg=9), SHAPE),
    (dict(best=0), SHAPE), (dict(best=3), SHAPE), (dict(g=64, kg=64, best=2), SHAPE), (dict(g=0), GROUP), (dict(g=7), GROUP),
    (dict(ld=3), DTYPE), (dict(sc=2), UNSUP), (dict(sc=-1), UNSUP), (dict(E=1032), UNSUP), (dict(E=1024, k=33), UNSUP),
    (dict(E=1024, g=128, kg=64, k=4), UNSUP), (dict(lg=0), NULL), (dict(i=0), NULL), (dict(w=0), NULL),
    (dict(lg=P + 2), ALIGN), (dict(b=P + 2), ALIGN), (dict(i=P + 1), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(T=0, lg=0, b=0, i=0, w=0), OK),
])
def test_moe_route_rejects(kw, want):
    assert route(**kw) == want


def routed(X=P, xd=BF16, i=P, w=P, gu=P, gus=P, dn=P, ds=P, Y=P, yd=BF16, T=2, E=8, k=2, H=256, F=128, G=128, ws=P,
           wb=1 << 40):
    return L.tern_moe_routed(X, xd, i, w, gu, gus, dn, ds, Y, yd, T, E, k, H, F, G, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(H=16384 + 128), SHAPE), (dict(H=192), GROUP),
    (dict(G=64), UNSUP), (dict(E=1025), UNSUP), (dict(k=33), UNSUP), (dict(xd=F32), DTYPE), (dict(yd=4), DTYPE),
    (dict(X=0), NULL), (dict(i=0), NULL), (dict(w=0), NULL), (dict(gu=0), NULL), (dict(dn=0), NULL), (dict(Y=0), NULL),
    (dict(ws=0), NULL), (dict(i=P + 2), ALIGN), (dict(w=P + 1), ALIGN), (dict(X=P + 8), ALIGN), (dict(ws=P + 128), ALIGN),
    (dict(wb=0), SHAPE), (dict(T=0, X=0, i=0, w=0, Y=0, ws=0), OK),
])
def test_moe_routed_rejects(kw, want):
    assert routed(**kw) == want


def test_binding_refuses_host_tensors_types_and_shapes():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    codes, scales = torch.zeros((2, 256), dtype=torch.int8), torch.zeros((2, 1))
    packed, ws = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.float16)
    for call in (lambda: tern.rms_norm(x, None), lambda: tern.rms_norm_q8(x, None), lambda: tern.q8_quantize(x),
                 lambda: tern.q8_dequant(codes, scales), lambda: tern.matmul_q8(codes, scales, packed, ws),
                 lambda: tern.moe_route(x, 2), lambda: tern.rms_norm_into(x, None)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tern.rms_norm(x.double(), None), lambda: tern.q8_quantize(x.int()),
                 lambda: tern.matmul_q8(codes.int(), scales, packed, ws), lambda: tern.moe_route(x.double(), 2)):
        with pytest.raises(TypeError):
            call()
