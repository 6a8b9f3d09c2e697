"""The gated product, the product with int8 weights and the layer norm on a host
without a GPU: what they refuse (before any device call, on addresses that are
never followed), the sizes of their workspaces, and the 64-bit definitions that
the GPU tests compare with, against finite differences."""
import ctypes

import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
import gated_ref as gref  # noqa: E402
from test_block_host import INF, NAN, WS, P, differences  # noqa: E402


def ln(X=P[0], kind=B.IN_F32, res=P[1], gain=P[2], beta=P[3], eps=1e-6, H=P[4], Y=P[5], mean=P[6], rstd=P[7], Q=P[8],
       s=P[9], R=4, C=8):
    return B.lib().ternary_layernorm_quantize(X, kind, res, gain, beta, eps, H, Y, mean, rstd, Q, s, R, C, None)


def ln_bwd(dY=P[0], H=P[1], kind=B.IN_F32, gain=P[2], mean=P[3], rstd=P[4], dH=P[5], dX=P[6], dg=P[7], db=P[8], R=4, C=8,
           ws=P[9], n=WS):
    return B.lib().ternary_layernorm_backward(dY, H, kind, gain, mean, rstd, dH, dX, dg, db, R, C, ws, n, None)


def gated_bwd(dY=P[0], Z=P[1], kind=B.IN_F32, act=0, dZ=P[2], db=P[3], Q=P[4], s=P[5], R=4, C=8, ws=P[6], n=WS):
    return B.lib().ternary_gated_backward(dY, Z, kind, act, 1.0, 1.0, dZ, db, Q, s, R, C, ws, n, None)


def gated(A=P[0], W=P[1], rs=P[2], bias=P[3], act=0, Y=P[4], Z=P[5], kind=B.OUT_F32, M=100, N=8, K=16, ws=P[6], n=WS):
    return B.lib().ternary_gemm_s8_gated(A, W, rs, 1.0, 1.0, bias, act, Y, Z, kind, M, N, K, ws, n, None)


def s8s8(A=P[0], W=P[1], rs=P[2], cs=P[3], bias=P[4], act=0, res=P[5], Y=P[6], Z=P[7], kind=B.OUT_F32, M=1000, N=8, K=17,
         ws=P[8], n=WS):
    return B.lib().ternary_gemm_s8s8_epilogue(A, W, rs, cs, bias, act, res, Y, Z, kind, M, N, K, ws, n, None)


@pytest.mark.parametrize("call,names", [
    (ln, ("X", "gain", "H", "Q", "s")), (ln_bwd, ("dY", "H", "gain", "mean", "rstd", "dX", "dg")),
    (gated_bwd, ("dY", "Z", "dZ", "Q", "s")), (gated, ("A", "W", "rs", "Y")), (s8s8, ("A", "W", "rs", "Y"))])
def test_null_pointers(call, names):
    for name in names:
        assert call(**{name: None}) == B.ERR_NULL, name
    if call is ln:                            # the statistics go together
        assert ln(mean=None) == B.ERR_NULL and ln(rstd=None) == B.ERR_NULL


@pytest.mark.parametrize("call", [ln, ln_bwd, gated_bwd])
def test_kinds_and_sizes(call):
    for kind in (0, 3, -1):
        assert call(kind=kind) == B.ERR_KIND
    for R, C in ((0, 8), (4, 0), (-1, 8), (4, -8), (1 << 40, 1 << 40), (1, 1 << 50)):
        assert call(R=R, C=C) == B.ERR_DIM, (R, C)


@pytest.mark.parametrize("call", [gated, s8s8])
def test_product_checks(call):
    for kind in (0, 3):
        assert call(kind=kind) == B.ERR_KIND
    for act in (-1, 5):
        assert call(act=act) == B.ERR_VALUE
    for M, N, K in ((0, 8, 16), (4, 0, 16), (4, 8, 0), (-4, 8, 16), (1 << 40, 1 << 40, 4), (4, (1 << 29) + 1, 4), (4, (1 << 27) + 1, 4), (1 << 36, 8, 4)):
        assert call(M=M, N=N, K=K) == B.ERR_DIM, (M, N, K)
    assert gated(K=18) == B.ERR_PACK and gated(K=16777220) == B.ERR_BOUND and s8s8(K=131072) == B.ERR_BOUND


def test_scalars_out_of_range():
    for eps in (-1e-6, NAN, INF):
        assert ln(eps=eps) == B.ERR_VALUE
    for act in (-1, 5):
        assert gated_bwd(act=act) == B.ERR_VALUE


def test_norm_aliases():
    n = 4 * 4 * 8
    for out in ("H", "Y", "Q", "s", "mean", "rstd"):
        for into in (P[0] + 4, P[1] + n - 1, P[2], P[3] + 28):
            assert ln(**{out: into}) == B.ERR_ALIAS, out
    assert ln(Y=P[4]) == B.ERR_ALIAS and ln(rstd=P[6] + 12) == B.ERR_ALIAS and ln(s=P[8] + 31) == B.ERR_ALIAS
    assert ln(Y=P[0]) == B.ERR_ALIAS               # in place is H's alone
    for out in ("dX", "dg", "db", "ws"):
        for into in (P[0], P[1], P[2], P[3], P[4]):
            assert ln_bwd(**{out: into}) == B.ERR_ALIAS, out
    assert ln_bwd(dX=P[5] + 16) == B.ERR_ALIAS and ln_bwd(dg=P[6]) == B.ERR_ALIAS and ln_bwd(db=P[7] + 4) == B.ERR_ALIAS


def test_gated_backward_aliases():
    for out in ("dZ", "db", "Q", "s", "ws"):
        for into in (P[0], P[1] + 4 * 4 * 16 - 1):   # Z's second half too
            assert gated_bwd(**{out: into}) == B.ERR_ALIAS, out
    assert gated_bwd(Q=P[2] + 4 * 4 * 16 - 4) == B.ERR_ALIAS and gated_bwd(db=P[4] + 63) == B.ERR_ALIAS
    assert gated_bwd(s=P[3] + 60) == B.ERR_ALIAS     # dbias has both halves


def test_product_aliases():
    for out in ("Y", "Z", "ws"):
        for into in (P[0] + 16, P[1], P[2], P[3] + 48):
            assert gated(**{out: into}) == B.ERR_ALIAS, out
        for into in (P[0] + 16, P[1], P[2], P[3], P[4] + 16, P[5] + 16):
            assert s8s8(**{out: into}) == B.ERR_ALIAS, out
    assert gated(Z=P[4]) == B.ERR_ALIAS and gated(Y=P[5] + 100 * 16 * 4 - 4) == B.ERR_ALIAS
    assert s8s8(Z=P[5]) == B.ERR_ALIAS and s8s8(Z=P[6]) == B.ERR_ALIAS and s8s8(ws=P[6] + 64) == B.ERR_ALIAS


def test_workspaces_of_the_backward_passes():
    b = ctypes.c_int64()
    for query, call in ((B.lib().ternary_layernorm_backward_workspace, ln_bwd), (B.lib().ternary_gated_backward_workspace, gated_bwd)):
        assert query(4, 8, None) == B.ERR_NULL and query(0, 8, ctypes.byref(b)) == B.ERR_DIM
        for R, C in ((1, 1), (27, 243), (16384, 3456), (3, 40000)):
            assert query(R, C, ctypes.byref(b)) == B.OK and 0 <= b.value <= 2 * (4 * 1024 * C + 4 * R + 1024)
        assert query(27, 243, ctypes.byref(b)) == B.OK and b.value == 0      # few short rows need none
        assert query(4000, 64, ctypes.byref(b)) == B.OK and b.value > 0
        kw = {"R": 4000, "C": 64}
        assert call(ws=None, **kw) == B.ERR_WORKSPACE and call(n=b.value - 1, **kw) == B.ERR_WORKSPACE
        assert call(ws=P[10] + 8, **kw) == B.ERR_WORKSPACE


def test_workspaces_of_the_products():
    b = ctypes.c_int64()
    g, s = B.lib().ternary_gemm_s8_gated_workspace, B.lib().ternary_gemm_s8s8_workspace

    def of(query, *args):
        assert query(*args, ctypes.byref(b)) == B.OK
        return b.value

    assert g(4, 8, 16, 16, None) == B.ERR_NULL and s(4, 8, 16, 16, None) == B.ERR_NULL
    assert g(0, 8, 16, 16, ctypes.byref(b)) == B.ERR_DIM and g(4, 8, 18, 16, ctypes.byref(b)) == B.ERR_PACK
    assert s(4, 8, 131072, 16, ctypes.byref(b)) == B.ERR_BOUND and g(4, 8, 16777220, 16, ctypes.byref(b)) == B.ERR_BOUND
    # few aligned rows run on the codes, others on the decoded weights, 2 N rows of whole 16-byte chunks
    assert of(g, 27, 100, 128, 16) == 0 and of(g, 27, 100, 128, 8) >= 2 * 100 * 128 + 27 * 128
    assert of(g, 27, 100, 132, 16) >= (2 * 100 + 27) * 144 and of(g, 5000, 100, 128, 256) == 2 * 100 * 128
    # few rows take any contraction as it lies; others need whole, aligned chunks
    assert of(s, 27, 100, 131, 1) == 0 and of(s, 5000, 100, 128, 16) == 0
    assert of(s, 5000, 100, 131, 16) >= 5100 * 144 and of(s, 5000, 100, 128, 1) >= 5100 * 128
    assert gated(ws=None) == B.ERR_WORKSPACE and gated(n=2 * 8 * 16 - 1) == B.ERR_WORKSPACE and gated(ws=P[6] + 8) == B.ERR_WORKSPACE
    assert s8s8(ws=None) == B.ERR_WORKSPACE and s8s8(n=1008 * 32 - 1) == B.ERR_WORKSPACE and s8s8(ws=P[8] + 8) == B.ERR_WORKSPACE


def test_wrappers_refuse_what_does_not_fit():
    host, q = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8)
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_layernorm_quantize(host, torch.ones(8))
    with pytest.raises(TypeError):
        B.ternary_layernorm_quantize(host.half(), torch.ones(8))
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_layernorm_backward(host, host, torch.ones(8), torch.ones(4), torch.ones(4))
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_gated_backward(host, host, 1.0, 1.0)
    with pytest.raises(TypeError):
        B.ternary_gated_backward(host, None, 1.0, 1.0)
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_gemm_s8s8_epilogue(q, q, torch.ones(4))
    with pytest.raises(TypeError):
        B.ternary_gemm_s8s8_epilogue(host, q, torch.ones(4))
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_gemm_s8_gated(q, torch.zeros(4, 2, dtype=torch.uint8), torch.ones(4), 1.0, 1.0)


# ---------------------------------------------------------------------------
# the definitions against finite differences
# ---------------------------------------------------------------------------

def test_layernorm_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    h, gain = torch.randn(3, 7, generator=g, dtype=torch.float64), torch.rand(7, generator=g, dtype=torch.float64) + 0.5
    beta = torch.randn(7, generator=g, dtype=torch.float64)
    dy, dH = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(2))
    f = lambda h, gain, beta: gref.layernorm(h, gain, beta, 1e-5)  # noqa: E731
    mean, _, rstd = f(h, gain, beta)[:3]
    dx, _, dg, _, db, _ = gref.layernorm_backward(dy, h, gain, mean, rstd, dH)
    assert torch.allclose(dx, differences(lambda v: (f(v, gain, beta)[4] * dy + v * dH).sum(), h), atol=1e-7)
    assert torch.allclose(dg, differences(lambda v: (f(h, v, beta)[4] * dy).sum(), gain), atol=1e-7)
    assert torch.allclose(db, differences(lambda v: (f(h, gain, v)[4] * dy).sum(), beta), atol=1e-7)


@pytest.mark.parametrize("act", B.ACTS)
def test_gated_gradients_against_differences(act):
    g = torch.Generator().manual_seed(2)
    Z = 2 * torch.randn(5, 12, generator=g, dtype=torch.float64)
    dy = torch.randn(5, 6, generator=g, dtype=torch.float64)
    zero = torch.zeros(5, 6, dtype=torch.float64)
    f = lambda z: (gref.gated(z[:, :6], zero, z[:, 6:], zero, act)[0] * dy).sum()  # noqa: E731
    dz, _, db, _ = gref.gated_backward(dy, Z, act)
    assert torch.allclose(dz, differences(f, Z), atol=1e-7) and torch.allclose(db, dz.sum(0))


def test_definitions_of_the_products():
    """The packed codes' order and the two halves, against sums written out."""
    g = torch.Generator().manual_seed(3)
    A = torch.randint(-128, 128, (3, 8), generator=g, dtype=torch.int8)
    W = torch.randint(0, 256, (4, 2), generator=g, dtype=torch.uint8)
    rs, bias = torch.rand(3, generator=g), torch.randn(4, generator=g)
    z, _, y, _ = gref.gated_product(A, W, rs, 0.5, 0.25, bias, "relu")
    for m in range(3):
        for n in range(2):
            v = []
            for row, scale in ((n, 0.5), (2 + n, 0.25)):
                acc = sum(int(A[m, k]) * (0, 1, -1, 0)[int(W[row, k // 4]) >> 2 * (k % 4) & 3] for k in range(8))
                v.append(acc * float(rs[m]) * scale + float(bias[row]))
            assert abs(float(z[m, n]) - v[0]) < 1e-5 and abs(float(z[m, 2 + n]) - v[1]) < 1e-5
            assert abs(float(y[m, n]) - max(v[0], 0) * v[1]) < 1e-4
    W8, cs = torch.randint(-128, 128, (2, 8), generator=g, dtype=torch.int8), torch.rand(2, generator=g)
    z, _, y, _ = gref.int8_product(A, W8, rs, cs, None, "relu2", torch.ones(3, 2))
    for m in range(3):
        for n in range(2):
            v = sum(int(A[m, k]) * int(W8[n, k]) for k in range(8)) * float(rs[m]) * float(cs[n])
            assert abs(float(z[m, n]) - v) < 1e-6 * abs(v) + 1e-9
            assert abs(float(y[m, n]) - max(v, 0) ** 2 - 1) < 1e-6 * v * v + 1e-6
    assert ref.U == 2.0 ** -24
