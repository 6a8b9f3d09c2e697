"""GPU parity of the gated product and of the product with int8 weights in every
kernel that their dispatch can choose (test_int8_plan.py holds the sizes to that):
each tile over several tiles a workgroup, whole and ragged ones, steps fewer and more
than its stages, with and without Z and residual, both kinds of activation."""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
import gated_ref as gref  # noqa: E402
from test_gpu_block import DEV, KINDS, gen, normal, say  # noqa: E402
from test_gpu_int8_products import int8, packed  # noqa: E402

pytestmark = pytest.mark.gpu

# (M, N, K)
INT8_TILES = [(788, 7593, 64), (883, 8381, 832), (1405, 8553, 528), (2385, 4883, 656), (7267, 2859, 736), (7413, 1673, 400),
              (8249, 604, 448), (8541, 390, 688)]
GATED_TILES = [(262, 8484, 176), (324, 8344, 800), (554, 8614, 800), (740, 8226, 400), (859, 6224, 400), (5466, 340, 592),
               (6029, 1795, 400)]
INT8_FEW = [(M, N, K) for M in (3, 27) for N, K in ((16401, 300), (8203, 520), (701, 1000), (702, 2600))]
GATED_FEW = [(M, N, 320) for M in (1, 7, 9, 16, 27, 70) for N in (100, 3456, 5002)]


def acts(i):
    return ("none", "relu", "relu2")[i % 3], ("silu", "gelu_tanh")[i % 2]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", INT8_TILES + INT8_FEW)
def test_int8_weights(M, N, K, kind):
    dt, g = KINDS[kind], gen("s8s8 kernels", M, N, K, kind)
    A, W, rs = int8(g, M, K), int8(g, N, K), 0.01 + torch.rand(M, generator=g, device=DEV)
    cs, bias = (0.5 + torch.rand(N, generator=g, device=DEV)) / (5000 * K ** 0.5), normal(g, N)
    res = normal(g, M, N, dtype=dt)
    for i, (save, r) in enumerate(((False, None), (True, None), (False, res), (True, res))):
        for act in acts(i):
            say(f"s8s8 {M}x{N}x{K} {kind} {act} save {save} residual {r is not None}")
            Y, Z = B.ternary_gemm_s8s8_epilogue(A, W, rs, cs, bias=bias, act=act, residual=r, out_dtype=dt, save=save)
            z, ez, y, ey = gref.int8_product(A, W, rs, cs, bias, act, r)
            ref.check(Y, y, ref.rounded(y, ey, dt), "Y")
            if save:
                ref.check(Z, z, ref.rounded(z, ez, dt), "Z")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", GATED_TILES + GATED_FEW)
def test_gated(M, N, K, kind):
    dt, g = KINDS[kind], gen("gated kernels", M, N, K, kind)
    A, W, rs = int8(g, M, K), packed(g, 2 * N, K), 0.01 + torch.rand(M, generator=g, device=DEV)
    gs, us, bias = float(torch.tensor(0.7 / K ** 0.5 / 40)), float(torch.tensor(0.02)), normal(g, 2 * N)
    for i, save in enumerate((False, True)):
        for act in acts(i + M):
            say(f"gated {M}x{N}x{K} {kind} {act} save {save}")
            Y, Z = B.ternary_gemm_s8_gated(A, W, rs, gs, us, bias=bias, act=act, out_dtype=dt, save=save)
            z, ez, y, ey = gref.gated_product(A, W, rs, gs, us, bias, act)
            ref.check(Y, y, ref.rounded(y, ey, dt), "Y")
            if save:
                ref.check(Z, z, ref.rounded(z, ez, dt), "Z")
