"""The operators around the product on a host without a GPU: what they refuse
(before any device call, on addresses that are never followed), the sizes of
their workspaces, and the 64-bit definitions that the GPU tests compare with,
against finite differences."""
import ctypes

import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402

P = [(i + 1) << 32 for i in range(12)]      # distinct addresses far apart
WS = 1 << 28
INF, NAN = float("inf"), float("nan")


def norm(X=P[0], kind=B.IN_F32, res=P[1], gain=P[2], eps=1e-6, H=P[3], Y=P[4], rstd=P[5], Q=P[6], s=P[7], R=4, C=8):
    return B.lib().ternary_rmsnorm_quantize(X, kind, res, gain, eps, H, Y, rstd, Q, s, R, C, None)


def norm_bwd(dY=P[0], H=P[1], kind=B.IN_F32, gain=P[2], rstd=P[3], dH=P[4], dX=P[5], dg=P[6], R=4, C=8, ws=P[7], n=WS):
    return B.lib().ternary_rmsnorm_backward(dY, H, kind, gain, rstd, dH, dX, dg, R, C, ws, n, None)


def product(A=P[0], W=P[1], rs=P[2], bias=P[3], act=0, res=P[4], Y=P[5], Z=P[6], kind=B.OUT_F32, M=4, N=8, K=16):
    return B.lib().ternary_gemm_s8_epilogue(A, W, rs, 1.0, bias, act, res, Y, Z, kind, M, N, K, None)


def epi_bwd(dY=P[0], Z=P[1], kind=B.IN_F32, act=0, dZ=P[2], db=P[3], Q=P[4], s=P[5], R=4, C=8, ws=P[6], n=WS):
    return B.lib().ternary_epilogue_backward(dY, Z, kind, act, dZ, db, Q, s, R, C, ws, n, None)


def clip(grads=(P[0], P[1]), outs=(P[2], P[3]), sizes=(8, 16), kinds=(1, 2), max_norm=1.0, eps=1e-6, norm_=P[4], ws=P[5],
         n=WS, count=None):
    k = len(sizes)
    arr = lambda t, v: (t * k)(*v)  # noqa: E731
    return B.lib().ternary_clip_grad_norm(arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs),
                                          arr(ctypes.c_int64, sizes), arr(ctypes.c_int32, kinds),
                                          k if count is None else count, max_norm, eps, norm_, ws, n, None)


@pytest.mark.parametrize("call,names", [
    (norm, ("X", "gain", "H", "Q", "s")), (norm_bwd, ("dY", "H", "gain", "rstd", "dX", "dg")),
    (product, ("A", "W", "rs", "Y")), (epi_bwd, ("dY", "Z", "dZ", "Q", "s")), (clip, ("norm_",))])
def test_null_pointers(call, names):
    for name in names:
        assert call(**{name: None}) == B.ERR_NULL, name


@pytest.mark.parametrize("call", [norm, norm_bwd, epi_bwd])
def test_kinds_and_sizes(call):
    for kind in (0, 3, -1):
        assert call(kind=kind) == B.ERR_KIND
    for R, C in ((0, 8), (4, 0), (-1, 8), (4, -8), (1 << 40, 1 << 40), (1, 1 << 50)):
        assert call(R=R, C=C) == B.ERR_DIM, (R, C)


def test_product_checks():
    for kind in (0, 3):
        assert product(kind=kind) == B.ERR_KIND
    for act in (-1, 5):
        assert product(act=act) == B.ERR_VALUE
    for M, N, K in ((0, 8, 16), (4, 0, 16), (4, 8, 0), (1 << 40, 1 << 40, 4)):
        assert product(M=M, N=N, K=K) == B.ERR_DIM
    assert product(K=18) == B.ERR_PACK
    assert product(K=B.lib() and 16777216 + 4) == B.ERR_BOUND


def test_scalars_out_of_range():
    for eps in (-1e-6, NAN, INF):
        assert norm(eps=eps) == B.ERR_VALUE
    for act in (-1, 5):
        assert epi_bwd(act=act) == B.ERR_VALUE
    for kw in ({"max_norm": -1.0}, {"max_norm": NAN}, {"eps": -1.0}, {"eps": NAN}):
        assert clip(**kw) == B.ERR_VALUE


def test_norm_aliases():
    n = 4 * 4 * 8
    for out in ("H", "Y", "Q", "s", "rstd"):
        for into in (P[0] + 4, P[1] + n - 1, P[2]):
            assert norm(**{out: into}) == B.ERR_ALIAS, out
    assert norm(Y=P[3]) == B.ERR_ALIAS and norm(Q=P[4] + 8) == B.ERR_ALIAS and norm(s=P[5]) == B.ERR_ALIAS
    assert norm(Y=P[0]) == B.ERR_ALIAS             # in place is H's alone


def test_backward_aliases():
    for out in ("dX", "dg", "ws"):
        for into in (P[0], P[1], P[2], P[3]):
            assert norm_bwd(**{out: into}) == B.ERR_ALIAS, out
    assert norm_bwd(dX=P[4] + 16) == B.ERR_ALIAS and norm_bwd(dg=P[5]) == B.ERR_ALIAS and norm_bwd(ws=P[6]) == B.ERR_ALIAS
    for out in ("dZ", "db", "Q", "s", "ws"):
        for into in (P[0], P[1]):
            assert epi_bwd(**{out: into}) == B.ERR_ALIAS, out
    assert epi_bwd(Q=P[2]) == B.ERR_ALIAS and epi_bwd(ws=P[4]) == B.ERR_ALIAS


def test_product_aliases():
    for into in (P[0] + 4, P[1], P[2], P[3], P[4] + 4):
        assert product(Y=into) == B.ERR_ALIAS and product(Z=into) == B.ERR_ALIAS
    assert product(Z=P[4]) == B.ERR_ALIAS and product(Z=P[5] + 64) == B.ERR_ALIAS


def test_workspaces():
    b = ctypes.c_int64()
    for query, call in ((B.lib().ternary_rmsnorm_backward_workspace, norm_bwd),
                        (B.lib().ternary_epilogue_backward_workspace, epi_bwd)):
        assert query(4, 8, None) == B.ERR_NULL and query(0, 8, ctypes.byref(b)) == B.ERR_DIM
        for R, C in ((1, 1), (27, 243), (16384, 3456), (3, 40000)):
            assert query(R, C, ctypes.byref(b)) == B.OK and 0 <= b.value <= 4 * 1024 * C + 4 * R + 1024
        assert query(4000, 64, ctypes.byref(b)) == B.OK and b.value > 0
        kw = {"R": 4000, "C": 64}
        assert call(ws=None, **kw) == B.ERR_WORKSPACE and call(n=b.value - 1, **kw) == B.ERR_WORKSPACE
        assert call(ws=P[9] + 8, **kw) == B.ERR_WORKSPACE
    q = B.lib().ternary_clip_grad_norm_workspace
    sizes = (ctypes.c_int64 * 3)(5, 0, 1 << 24)
    assert q(sizes, 3, ctypes.byref(b)) == B.OK and b.value > 16
    assert q(None, 3, ctypes.byref(b)) == B.ERR_NULL and q(sizes, 3, None) == B.ERR_NULL
    assert q(sizes, 0, ctypes.byref(b)) == B.ERR_DIM
    assert q((ctypes.c_int64 * 1)(-1), 1, ctypes.byref(b)) == B.ERR_DIM
    assert q((ctypes.c_int64 * 2)(1 << 62, 1 << 62), 2, ctypes.byref(b)) == B.ERR_DIM
    assert clip(ws=None) == B.ERR_WORKSPACE and clip(n=8) == B.ERR_WORKSPACE and clip(ws=P[5] + 8) == B.ERR_WORKSPACE


def test_clip_lists():
    assert clip(count=0) == B.ERR_DIM and clip(sizes=(-1, 16)) == B.ERR_DIM
    assert clip(grads=(P[0], None)) == B.ERR_NULL and clip(outs=(None, P[3])) == B.ERR_NULL
    assert clip(kinds=(1, 0)) == B.ERR_KIND
    assert clip(norm_=P[0]) == B.ERR_ALIAS and clip(norm_=P[3] + 4) == B.ERR_ALIAS and clip(norm_=P[5]) == B.ERR_ALIAS
    assert clip(ws=P[1]) == B.ERR_ALIAS and clip(ws=P[2]) == B.ERR_ALIAS
    assert clip(outs=(P[0] + 4, P[3])) == B.ERR_ALIAS      # its own gradient, shifted
    assert clip(outs=(P[1] + 4, P[3])) == B.ERR_ALIAS      # another's gradient
    assert clip(outs=(P[2], P[2] + 16)) == B.ERR_ALIAS     # each other
    assert clip(outs=(P[1], P[0])) == B.ERR_ALIAS          # exchanged
    assert clip(grads=(P[0], P[0]), outs=(P[0], P[0])) == B.ERR_ALIAS   # one gradient listed twice, in place


def test_wrappers_refuse_what_does_not_fit():
    host = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_rmsnorm_quantize(host, torch.ones(8))
    with pytest.raises(TypeError):
        B.ternary_rmsnorm_quantize(host.half(), torch.ones(8))
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_rmsnorm_backward(host, host, torch.ones(8), torch.ones(4))
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_epilogue_backward(host, host)
    with pytest.raises(ValueError, match="device tensor"):
        B.ternary_gemm_s8_epilogue(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8), torch.ones(4), 1.0)
    with pytest.raises(ValueError, match="device"):
        B.ternary_clip_grad_norm([host], 1.0)
    with pytest.raises(ValueError, match="at least one"):
        B.ternary_clip_grad_norm([], 1.0)
    with pytest.raises(TypeError):
        B.ternary_clip_grad_norm([host.double()], 1.0)


# ---------------------------------------------------------------------------
# the definitions against finite differences
# ---------------------------------------------------------------------------

def differences(f, x, h=1e-6):
    """df/dx of a scalar f by central differences, element by element."""
    d = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        d.view(-1)[i] = (f(x + e.view_as(x)) - f(x - e.view_as(x))) / (2 * h)
    return d


def test_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    h, gain = torch.randn(3, 7, generator=g, dtype=torch.float64), torch.rand(7, generator=g, dtype=torch.float64) + 0.5
    dy, dH = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(2))
    rstd = ref.norm(h, gain, 1e-5)[0]
    dx, _, dg, _ = ref.norm_backward(dy, h, gain, rstd, dH)
    assert torch.allclose(dx, differences(lambda v: (ref.norm(v, gain, 1e-5)[2] * dy + v * dH).sum(), h), atol=1e-7)
    assert torch.allclose(dg, differences(lambda v: (ref.norm(h, v, 1e-5)[2] * dy).sum(), gain), atol=1e-7)


@pytest.mark.parametrize("act", B.ACTS)
def test_activation_slopes_against_differences(act):
    z = torch.linspace(-9.05, 9.05, 182, dtype=torch.float64)
    d = differences(lambda v: ref.activation(v, torch.zeros_like(v), act)[0].sum(), z)
    assert torch.allclose(ref.slope(z, act)[0], d, atol=1e-6)
    dy = torch.linspace(-1, 1, 182, dtype=torch.float64).view(14, 13)
    dz, _, db, _ = ref.epilogue_backward(dy, z.view(14, 13), act)
    assert torch.allclose(dz, dy * d.view(14, 13), atol=1e-6) and torch.allclose(db, dz.sum(0))
